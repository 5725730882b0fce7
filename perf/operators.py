"""The measured cases of the attention operators: the full-attention layers of the hybrid
stack, which sit between the Gated DeltaNet layers.

Four operators, as a serving program calls them around one paged key-value cache:

* ``append``  -- rotate the new tokens' queries and keys by their positions, write keys and
  values into the cache's pages, return the rotated queries;
* ``decode``  -- one new token per sequence attends to its sequence's pages;
* ``prefill`` -- whole prompts, causal, grouped heads, dense or packed;
* ``paged``   -- prompt pieces attend to the cache that holds their past and themselves.

The plain forms are elementary torch operations in 32 bits (angles in 64); ``exact`` is the
definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, **kw):
    base = dict(name=name, op=op, dtype="bf16", hq=32, hkv=8, d=128, page=64, seqs=1, lo=1, hi=1, past_lo=0,
                past_hi=0, rotary=0, interleaved=False, fused=False, gate=False, dense=False, idle=0, lens=1)
    base.update(kw)
    return base


def listed():
    return [
        # one decode step of a serving batch: the smallest call, all launch latency
        _case("append_step_b64", "append", seqs=64, lo=1, hi=1, past_lo=100, past_hi=8000, rotary=64, fused=True),
        # a packed batch of prompts entering the cache straight from the fused projection
        _case("append_prompts_32k", "append", seqs=11, lo=512, hi=5446, rotary=128, fused=True, page=64),
        # pieces of odd length in fp32, 64-wide heads, interleaved pairs, far positions
        _case("append_pieces_fp32", "append", dtype="fp32", hq=8, hkv=8, d=64, page=16, seqs=3, lo=700, hi=1801,
              past_lo=90000, past_hi=262144, rotary=64, interleaved=True),
        # one user, a short chat: latency of a single call
        _case("decode_b1_short", "decode", seqs=1, lo=1000, hi=1000, page=16),
        # the serving batch of the decode workload with ragged contexts and gated outputs
        _case("decode_b64_ragged", "decode", seqs=64, lo=17, hi=32768, gate=True),
        # one user far into a long document, few key-value heads: the length is all there is to split
        _case("decode_b1_long", "decode", seqs=1, lo=262143, hi=262143, hq=16, hkv=2, page=128),
        # fp32, no grouping, 64-wide heads, a batch with idle slots
        _case("decode_fp32_d64", "decode", dtype="fp32", hq=16, hkv=16, d=64, page=32, seqs=24, lo=1, hi=4000, idle=3),
        # a packed batch of prompts, 512 to 8,192 tokens each, about 65,000 in all
        _case("prefill_packed_64k", "prefill", seqs=15, lo=512, hi=8192, gate=True),
        # one long prompt
        _case("prefill_long_32k", "prefill", seqs=1, lo=32768, hi=32768, hq=16, hkv=4),
        # a dense batch in fp32 with 64-wide heads
        _case("prefill_fp32_dense", "prefill", dtype="fp32", hq=8, hkv=2, d=64, seqs=3, lo=1111, hi=1111, dense=True),
        # prompt pieces over long pasts
        _case("paged_pieces", "paged", seqs=4, lo=1500, hi=2500, past_lo=2000, past_hi=30000, gate=True),
        # a few tokens a sequence (drafts to be verified) over long pasts: little to do a row, long rows
        _case("paged_drafts", "paged", seqs=8, lo=2, hi=40, past_lo=3000, past_hi=16000, page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "paged"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([128, 128, 64])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]) if hkv <= 2 else rng.choice([1, 2, 3, 4])
    page = rng.choice([16, 32, 64, 128])
    kw = dict(dtype=dtype, d=d, hkv=hkv, hq=hkv * group, page=page, lens=rng.randrange(1 << 30),
              gate=rng.random() < 0.5)
    cap = 2048 if dtype == "fp32" else 12000
    if op == "append":
        seqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, 24000 // seqs))
        past = _log_int(rng, 1, 60000)
        kw.update(gate=False, seqs=seqs, lo=max(1, hi // 3), hi=hi, past_lo=0, past_hi=min(past, 250000 // seqs),
                  rotary=rng.choice([0, d // 4, d // 2, d]), interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
    elif op == "decode":
        seqs = _log_int(rng, 1, 160)
        hi = _log_int(rng, 1, min(200000, (900000 if dtype == "bf16" else 450000) // seqs))
        kw.update(seqs=seqs, lo=max(1, hi // rng.choice([1, 4, 50])), hi=hi, idle=rng.choice([0, 0, 2]))
    elif op == "prefill":
        hi = _log_int(rng, 1, cap)
        seqs = _log_int(rng, 1, max(1, min(40, 30000 // hi)))
        kw.update(seqs=seqs, lo=max(1, hi // 4), hi=hi, dense=rng.random() < 0.3)
    else:
        seqs = _log_int(rng, 1, 12)
        hi = _log_int(rng, 1, cap // seqs)
        past = _log_int(rng, 1, cap)
        kw.update(seqs=seqs, lo=max(1, hi // 3), hi=hi, past_lo=past // 3, past_hi=past)
    c = _case("", op, **kw)
    del c["name"]
    return c


def _lens(case):
    """(new tokens of each sequence, tokens each holds in the cache before them), from the case alone."""
    r = random.Random(case["lens"] * 7919 + case["seqs"])
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    if case["dense"]:
        new = [case["hi"]] * case["seqs"]
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])]
    if case["op"] == "decode":              # `lo`..`hi` are context lengths, the new token among them
        past, new = [n - 1 for n in new], [1] * case["seqs"]
        for i in range(case["idle"]):       # idle slots of a padded batch: no context at all
            past[(i * 5 + 1) % case["seqs"]] = -1
    return new, past


def work(case):
    new, past = _lens(case)
    es, hq, hkv, d = _ES[case["dtype"]], case["hq"], case["hkv"], case["d"]
    T = sum(new)
    if case["op"] == "append":
        table = sum(-(-(n + p) // case["page"]) - p // case["page"] for n, p in zip(new, past)) * 4
        return {"bytes": T * (2 * hq + 4 * hkv) * d * es + table + case["rotary"] * 2,
                "flops": T * (hq + hkv) * case["rotary"] * 3}
    rows = 2 + (1 if case["gate"] else 0)
    if case["op"] == "decode":
        ctx = sum(p + 1 for p in past)
        table = sum(-(-(p + 1) // case["page"]) for p in past) * 4
        return {"bytes": ctx * 2 * hkv * d * es + T * rows * hq * d * es + table, "flops": 4 * ctx * hq * d}
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    keys = sum(n + p for n, p in zip(new, past))
    return {"bytes": keys * 2 * hkv * d * es + T * rows * hq * d * es, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _fill(gen, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (t * scale).to(dtype) if scale != 1.0 else t.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, hq, hkv, d, page = _DT[case["dtype"]], case["hq"], case["hkv"], case["d"], case["page"]
    new, past = _lens(case)
    T, N = sum(new), case["seqs"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=case, new=new, past=past, cu=cu, scale=d ** -0.5)
    s["cu_dev"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    # queries of some heads are sharper than others, as trained heads are
    sharp = torch.linspace(0.5, 2.5, hq, device="cuda")[None, :, None]
    if case["fused"]:                        # the fused projection's output, read through views
        x = _fill(gen, (T, (hq + 2 * hkv) * d), dt)
        s["q"], s["k"], s["v"] = (x[:, :hq * d].view(T, hq, d), x[:, hq * d:(hq + hkv) * d].view(T, hkv, d),
                                  x[:, (hq + hkv) * d:].view(T, hkv, d))
    else:
        s["q"] = (_fill(gen, (T, hq, d), torch.float32) * sharp).to(dt)
        if case["op"] in ("append", "prefill"):
            s["k"], s["v"] = _fill(gen, (T, hkv, d), dt), _fill(gen, (T, hkv, d), dt)
    if case["gate"]:
        s["z"] = _fill(gen, (T, hq, d), dt)
    else:
        s["z"] = None
    if case["op"] == "prefill":
        if case["dense"]:
            B, L = N, new[0]
            for key in ("q", "k", "v", "z"):
                if s[key] is not None:
                    s[key] = s[key].view(B, L, *s[key].shape[1:])
        else:
            for key in ("q", "k", "v", "z"):
                if s[key] is not None:
                    s[key] = s[key].unsqueeze(0)
        s["o"] = torch.empty_like(s["q"])
    else:
        # pages are handed out in no order; entries past a sequence's end hold -1
        total = [n + p for n, p in zip(new, past)]
        need = [-(-t // page) for t in total]
        n_pages, width = sum(need) + 3, max(max(need), 1)
        perm = torch.randperm(n_pages, generator=gen, device="cuda").tolist()
        table = np.full((N, width), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = perm[at:at + n]
            at += n
        s["table"] = torch.from_numpy(table).cuda()
        s["kv_lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        s["k_cache"] = _fill(gen, (n_pages, page, hkv, d), dt)
        s["v_cache"] = _fill(gen, (n_pages, page, hkv, d), dt)
        s["o"] = torch.empty((T, hq, d), dtype=dt, device="cuda")
    if case["op"] == "append":
        # where every token goes, as a scheduler knows it on the host
        pos = np.concatenate([np.arange(p, p + n) for n, p in zip(new, past)])
        seq = np.repeat(np.arange(N), new)
        slot = table[seq, pos // page].astype(np.int64) * page + pos % page
        s["pos"], s["slot"] = torch.from_numpy(pos).cuda(), torch.from_numpy(slot).cuda()
        s["inv_freq"] = None
        if case["rotary"]:
            r = torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64) / case["rotary"]
            s["inv_freq"] = (1e7 ** -r).float()
    if own and case["op"] != "append":
        import gated_deltanet_sequence_delta_b200 as G
        io = 1 if dt == torch.bfloat16 else 0
        if case["op"] == "decode":
            n = G.attn_decode_workspace_bytes(N, hq, hkv, d, io)
        else:
            n = G.attn_prefill_workspace_bytes(T, N, hq, hkv, d, io)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, rotary, interleaved):
    """x [T, H, D] fp32, cos and sin [T, 1, rotary / 2]."""
    if not rotary:
        return x
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rotary // 2], x[..., rotary // 2:rotary]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((r, x[..., rotary:]), dim=-1)


def _append_plain(s):
    c = s["case"]
    cos = sin = None
    if c["rotary"]:
        ang = s["pos"].double()[:, None, None] * s["inv_freq"].double()
        cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    q = _rotate(s["q"].float(), cos, sin, c["rotary"], c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, c["rotary"], c["interleaved"]).to(s["k"].dtype)
    s["k_cache"].view(-1, c["hkv"], c["d"])[s["slot"]] = k
    s["v_cache"].view(-1, c["hkv"], c["d"])[s["slot"]] = s["v"]
    s["o"].copy_(q)
    return s["o"], s["k_cache"], s["v_cache"]


def _attend_plain(q, k, v, past, scale):
    """q [n, HQ, D], k and v [n + past, HKV, D] in fp32: causal, the last query at the last key."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    g = hq // hkv
    kt, vt = k.permute(1, 2, 0), v.permute(1, 0, 2)                # [HKV, D, K], [HKV, K, D]
    out = torch.empty_like(q)
    step = max(16, min(n, (1 << 28) // (hq * k.shape[0])))
    for r0 in range(0, n, step):
        r1 = min(n, r0 + step)
        m = r1 - r0
        keys = past + r1
        qs = (q[r0:r1] * scale).view(m, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * m, d)
        sc = torch.matmul(qs, kt[:, :, :keys]).view(hkv, g, m, keys)
        row = torch.arange(past + r0, past + r1, device=q.device)[:, None]
        sc = sc.masked_fill_(torch.arange(keys, device=q.device)[None, :] > row, float("-inf"))
        sc = torch.exp(sc.sub_(sc.amax(dim=-1, keepdim=True)))
        den = sc.sum(dim=-1, keepdim=True)
        o = torch.matmul(sc.view(hkv, g * m, keys), vt[:, :keys]).view(hkv, g, m, d) / den
        out[r0:r1] = o.permute(2, 0, 1, 3).reshape(m, hq, d)
    return out


def _pages_of(s, i, total):
    """Keys and values of sequence i, in order, in fp32."""
    c = s["case"]
    idx = s["table"][i, :-(-total // c["page"])].long()
    k = s["k_cache"][idx].view(-1, c["hkv"], c["d"])[:total].float()
    v = s["v_cache"][idx].view(-1, c["hkv"], c["d"])[:total].float()
    return k, v


def _attention_plain(s):
    c = s["case"]
    shape = s["q"].shape
    q = s["q"].reshape(-1, c["hq"], c["d"])
    z = None if s["z"] is None else s["z"].reshape(q.shape)
    o = s["o"].view(q.shape)
    for i, (n, p) in enumerate(zip(s["new"], s["past"])):
        t0, t1 = s["cu"][i], s["cu"][i + 1]
        if c["op"] == "prefill":
            k = s["k"].reshape(-1, c["hkv"], c["d"])[t0:t1].float()
            v = s["v"].reshape(-1, c["hkv"], c["d"])[t0:t1].float()
        else:
            k, v = _pages_of(s, i, n + p)
        r = _attend_plain(q[t0:t1].float(), k, v, p, s["scale"])
        if z is not None:
            r = r / (1 + torch.exp(-z[t0:t1].float()))
        o[t0:t1] = r.to(o.dtype)
    return o.view(shape)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _append_plain(s) if op == "append" else _attention_plain(s)
    import gated_deltanet_sequence_delta_b200 as G
    if op == "append":
        G.gdn_attn_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                          cu_seqlens=s["cu_dev"], inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"],
                          q_out=s["o"])
        return s["o"], s["k_cache"], s["v_cache"]
    if op == "decode":
        return G.gdn_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], scale=s["scale"],
                                 z=s["z"], o=s["o"], workspace=s["ws"])
    if op == "paged":
        return G.gdn_attn_prefill_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu_dev"],
                                        scale=s["scale"], z=s["z"], o=s["o"], workspace=s["ws"])
    cu = None if s["case"]["dense"] else s["cu_dev"]
    return G.gdn_attn_prefill(s["q"], s["k"], s["v"], cu_seqlens=cu, scale=s["scale"], z=s["z"], o=s["o"],
                              workspace=s["ws"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        half = case["rotary"] // 2

        def turned(x):
            y = x.double().clone()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                w = torch.complex(y[..., a], y[..., b])
                ang = s["pos"].double() * float(s["inv_freq"][i].double())
                w = w * torch.polar(torch.ones_like(ang), ang)[:, None]
                y[..., a], y[..., b] = w.real, w.imag
            return y

        kc, vc = s["k_cache"].double().view(-1, hkv, d), s["v_cache"].double().view(-1, hkv, d)
        kc.index_copy_(0, s["slot"], turned(s["k"]))
        vc.index_copy_(0, s["slot"], s["v"].double().contiguous())
        return turned(s["q"]), kc.view(s["k_cache"].shape), vc.view(s["v_cache"].shape)
    q = s["q"].reshape(-1, hq, d)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for i, (n, p) in enumerate(zip(s["new"], s["past"])):
        total, t0 = n + p, s["cu"][i]
        if total <= 0:
            continue
        if case["op"] == "prefill":
            rows = torch.arange(t0, t0 + n, device="cuda")
            ks, vs = s["k"].reshape(-1, hkv, d), s["v"].reshape(-1, hkv, d)
        else:
            at = torch.arange(total, device="cuda")
            rows = s["table"][i].long()[at // case["page"]] * case["page"] + at % case["page"]
            ks, vs = s["k_cache"].view(-1, hkv, d), s["v_cache"].view(-1, hkv, d)
        for h in range(hq):
            kh, vh = ks[rows, h * hkv // hq].double(), vs[rows, h * hkv // hq].double()
            for r0 in range(0, n, 4096):
                r1 = min(n, r0 + 4096)
                qh = q[t0 + r0:t0 + r1, h].double()
                w = qh @ kh[:p + r1].T * s["scale"]
                w += torch.full_like(w, float("-inf")).triu_(p + r0 + 1)
                out[t0 + r0:t0 + r1, h] = torch.softmax(w, dim=-1) @ vh[:p + r1]
    if s["z"] is not None:
        out = out * torch.sigmoid(s["z"].reshape(q.shape).double())
    return out.view(s["q"].shape)
