"""The attention operators on the GPU against the fp64 definition (attn_ref), at the sizes and
masks where they can go wrong.  Bounds: attn_ref's, derived there."""
import numpy as np
import pytest

import attn_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "fp32": "float32"}


def _torch():
    import torch
    return torch, __import__("gated_deltanet_sequence_delta_b200")


def _draw(gen, shape, dtype, scale=1.0):
    torch, _ = _torch()
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(getattr(torch, DT[dtype]))


def _gen(seed):
    torch, _ = _torch()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    torch, _ = _torch()
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist()


def _close(got, want, bound, what):
    got = _np(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), (f"{what}: off by {np.abs(got - want).flat[over.argmax()]:.3e}, bound "
                               f"{bound.flat[over.argmax()]:.3e}, at {np.unravel_index(over.argmax(), over.shape)}")


class Cache:
    """A paged cache whose pages are handed out in no order; every slot that no sequence holds is
    NaN, and table entries past a sequence's end are -1."""

    def __init__(self, totals, HKV, D, page, dtype, seed, extra=2, v_scale=1.0):
        torch, _ = _torch()
        g = _gen(seed)
        need = [-(-t // page) for t in totals]
        self.page, self.totals = page, totals
        n = sum(need) + extra
        perm = torch.randperm(n, generator=g, device="cuda").tolist()
        self.table_np = np.full((len(totals), max(max(need), 1)), -1, dtype=np.int32)
        at = 0
        for i, c in enumerate(need):
            self.table_np[i, :c] = perm[at:at + c]
            at += c
        self.k = torch.full((n, page, HKV, D), float("nan"), dtype=getattr(torch, DT[dtype]), device="cuda")
        self.v = self.k.clone()
        self.table = torch.from_numpy(self.table_np).cuda()
        self.lens = _i32(totals)
        for i, t in enumerate(totals):
            if t:
                s = self.slots(i, 0, t)
                self.k.view(-1, HKV, D)[s] = _draw(g, (t, HKV, D), dtype)
                self.v.view(-1, HKV, D)[s] = _draw(g, (t, HKV, D), dtype, v_scale)

    def slots(self, i, p0, p1):
        torch, _ = _torch()
        pos = np.arange(p0, p1)
        return torch.from_numpy(self.table_np[i, pos // self.page].astype(np.int64) * self.page + pos % self.page).cuda()

    def seq(self, i):
        HKV, D = self.k.shape[2:]
        s = self.slots(i, 0, self.totals[i])
        return _np(self.k.view(-1, HKV, D)[s]), _np(self.v.view(-1, HKV, D)[s])


# ---- append -----------------------------------------------------------------------------
APPEND = [
    # dtype, D, HQ, HKV, page, rotary, interleaved, fused, new, past
    ("bf16", 128, 8, 2, 16, 128, False, True, [1, 0, 40, 17], [0, 5, 15, 1000]),
    ("bf16", 128, 4, 4, 64, 32, False, False, [300], [261000]),
    ("bf16", 64, 6, 2, 32, 64, True, True, [5, 33], [31, 32]),
    ("bf16", 64, 1, 1, 128, 0, False, False, [129, 1], [0, 127]),
    ("bf16", 128, 16, 1, 16, 16, True, False, [3, 3, 3], [7, 8, 9]),
    ("fp32", 64, 5, 5, 16, 64, True, False, [18, 1], [262143, 0]),
    ("fp32", 128, 8, 2, 64, 96, False, True, [70], [100]),
    ("fp32", 128, 2, 1, 32, 16, False, False, [1100], [3]),
]


@pytest.mark.parametrize("dtype,D,HQ,HKV,page,rotary,il,fused,new,past", APPEND)
def test_append(dtype, D, HQ, HKV, page, rotary, il, fused, new, past):
    torch, G = _torch()
    g = _gen(sum(new) + D)
    T, cu = sum(new), _cu(new)
    totals = [n + p for n, p in zip(new, past)]
    c = Cache(totals, HKV, D, page, dtype, 3)
    if fused:
        x = _draw(g, (T, (HQ + 2 * HKV) * D + 16), dtype)[:, :(HQ + 2 * HKV) * D]
        q, k, v = (x[:, :HQ * D].unflatten(1, (HQ, D)), x[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D)),
                   x[:, (HQ + HKV) * D:].unflatten(1, (HKV, D)))
    else:
        q, k, v = _draw(g, (T, HQ, D), dtype), _draw(g, (T, HKV, D), dtype), _draw(g, (T, HKV, D), dtype)
    f = None
    if rotary:
        f = (1e6 ** -(torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)).float()
    kc0, vc0 = c.k.clone(), c.v.clone()
    qo = G.gdn_attn_append(q, k, v, c.k, c.v, c.table, c.lens, cu_seqlens=_i32(cu), inv_freq=f, interleaved=il)
    fn = np.zeros(0) if f is None else _np(f)
    written = torch.zeros(c.k.shape[0] * page, dtype=torch.bool, device="cuda")
    probe = np.random.default_rng(0)
    for i, n in enumerate(new):
        if n == 0:
            continue
        s = c.slots(i, past[i], totals[i])
        written[s] = True
        kk, vv = c.k.view(-1, HKV, D)[s], c.v.view(-1, HKV, D)[s]
        assert torch.equal(vv, v[cu[i]:cu[i + 1]])
        rows = sorted({0, n - 1, *probe.integers(0, n, 6).tolist()})
        for src, got, H in ((q, qo[cu[i]:cu[i + 1]], HQ), (k, kk, HKV)):
            for t in rows:
                for h in {0, H - 1, H // 2}:
                    xin = _np(src[cu[i] + t, h])
                    want = R.rotate(xin, past[i] + t, fn, il)
                    _close(got[t, h], want, R.rotate_bound(xin, want, fn, il, dtype), f"seq {i} token {t} head {h}")
    # nothing else in the cache has moved (bit for bit, NaN included)
    for now, was in ((c.k, kc0), (c.v, vc0)):
        bits = lambda t: t.view(-1, HKV * D).view(torch.int16 if dtype == "bf16" else torch.int32)
        assert torch.equal(bits(now)[~written], bits(was)[~written])
    assert G.gdn_attn_status() == 0


def test_append_in_place_without_queries_and_idle_slots():
    torch, G = _torch()
    g = _gen(5)
    c = Cache([5, 0, 20], 2, 128, 16, "bf16", 1)
    q, k, v = _draw(g, (3, 4, 128), "bf16"), _draw(g, (3, 2, 128), "bf16"), _draw(g, (3, 2, 128), "bf16")
    f = torch.rand(64, device="cuda")
    want = torch.full_like(q, 7.0)
    a = (k, v, c.k, c.v, c.table, c.lens)
    G.gdn_attn_append(q, *a, inv_freq=f, q_out=want)
    assert (want[1] == 7.0).all()                       # an idle slot's row is left as it was
    kc, vc = c.k.clone(), c.v.clone()
    q2 = q.clone()
    assert G.gdn_attn_append(q2, *a, inv_freq=f, q_out=q2) is q2
    assert torch.equal(q2[[0, 2]], want[[0, 2]]) and torch.equal(q2[1], q[1])
    c.k.fill_(float("nan")), c.v.fill_(float("nan"))
    assert G.gdn_attn_append(None, *a, inv_freq=f) is None
    s = torch.cat([c.slots(0, 4, 5), c.slots(2, 19, 20)])
    for now, was in ((c.k, kc), (c.v, vc)):
        assert torch.equal(now.view(-1, 256)[s], was.view(-1, 256)[s])
        assert torch.isnan(now).sum() == now.numel() - 2 * 256
    assert G.gdn_attn_status() == 0


def test_append_far_positions():
    """fp32 angles at positions where their fp32 product would be off by 2^-5 rad."""
    torch, G = _torch()
    g = _gen(6)
    past = [1 << 19, (1 << 19) + 12345, (1 << 20) - 1]
    page, width = 128, ((1 << 20) >> 7) + 1
    q, k, v = _draw(g, (3, 1, 64), "fp32"), _draw(g, (3, 1, 64), "fp32"), _draw(g, (3, 1, 64), "fp32")
    f = torch.linspace(1.0, 0.1, 32, device="cuda")
    table = torch.zeros((3, width), dtype=torch.int32, device="cuda")
    for i, p in enumerate(past):
        table[i, p // page] = i
    kc = torch.zeros((3, page, 1, 64), device="cuda")
    qo = G.gdn_attn_append(q, k, v, kc, kc.clone(), table, _i32([p + 1 for p in past]), inv_freq=f)
    for i, p in enumerate(past):
        for got, src in ((qo[i, 0], q[i, 0]), (kc[i, p % page, 0], k[i, 0])):
            want = R.rotate(_np(src), p, _np(f), False)
            _close(got, want, R.rotate_bound(_np(src), want, _np(f), False, "fp32"), f"position {p}")


# ---- prompts -------------------------------------------------------------------------
def _check_rows(o, q, k, v, past, scale, dtype, z, what, rows=None):
    n = q.shape[0]
    rows = range(n) if rows is None else rows
    for i in rows:
        m = max(past + i + 1, 0)
        want, bound = R.attention(_np(q[i:i + 1]), k[:m], v[:m], m - 1, scale, dtype,
                                  None if z is None else _np(z[i:i + 1]))
        _close(o[i:i + 1], want, bound, f"{what} row {i}")


def _some(n, seed, count=24):
    """Rows to compare: the ends, those around tile borders, some at random."""
    r = np.random.default_rng(seed)
    edge = {0, 1, n - 1, n - 2, 31, 32, 63, 64, 127, 128, 129, 255, 256, 257}
    return sorted(i for i in edge | set(r.integers(0, max(n, 1), count).tolist()) if 0 <= i < n)


PREFILL = [
    # dtype, D, HQ, HKV, lengths, gate
    ("bf16", 128, 4, 2, [1, 2, 0, 63, 64, 65, 127, 128, 129], True),
    ("bf16", 128, 2, 1, [255, 256, 257], False),
    ("bf16", 128, 8, 8, [300], True),
    ("bf16", 128, 16, 1, [130, 7], False),
    ("bf16", 64, 6, 2, [200, 1, 129], True),
    ("bf16", 64, 3, 1, [513], False),
    ("bf16", 128, 4, 4, [1000, 3, 700], False),
    ("bf16", 64, 10, 2, [2100], True),
    ("fp32", 128, 4, 2, [1, 64, 65, 0, 130], True),
    ("fp32", 64, 6, 2, [257, 3], False),
    ("fp32", 128, 5, 1, [100], False),
    ("fp32", 64, 16, 1, [90], True),
]


@pytest.mark.parametrize("dtype,D,HQ,HKV,lens,gate", PREFILL)
def test_prefill_packed(dtype, D, HQ, HKV, lens, gate):
    torch, G = _torch()
    g = _gen(11)
    T, cu = sum(lens), _cu(lens)
    behind = 5                                           # rows behind the last sequence
    q = _draw(g, (1, T + behind, HQ, D), dtype, 1.5)
    k, v = _draw(g, (1, T + behind, HKV, D), dtype), _draw(g, (1, T + behind, HKV, D), dtype)
    z = _draw(g, (1, T + behind, HQ, D), dtype) if gate else None
    o = torch.full_like(q, 7.0)
    G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32(cu), z=z, o=o)
    kn, vn = _np(k[0]), _np(v[0])
    for i, n in enumerate(lens):
        a, b = cu[i], cu[i + 1]
        _check_rows(o[0, a:b], q[0, a:b], kn[a:b], vn[a:b], 0, D ** -0.5, dtype, None if z is None else z[0, a:b],
                    f"sequence {i}", _some(n, i))
    assert (o[0, T:] == 7.0).all()
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T", [(3, 100), (2, 257), (1, 1)])
def test_prefill_dense(dtype, B, T):
    torch, G = _torch()
    g = _gen(12)
    q, k, v = _draw(g, (B, T, 4, 128), dtype), _draw(g, (B, T, 2, 128), dtype), _draw(g, (B, T, 2, 128), dtype)
    o = G.gdn_attn_prefill(q, k, v, scale=0.2)
    for b in range(B):
        _check_rows(o[b], q[b], _np(k[b]), _np(v[b]), 0, 0.2, dtype, None, f"batch {b}", _some(T, b, 8))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_growing_and_sharp_scores(dtype):
    """Keys that grow along the sequence, so that the running maximum rises in every step, and
    scores of a few hundred, so that one key takes nearly all the weight."""
    torch, G = _torch()
    g = _gen(13)
    T = 700
    q, k, v = _draw(g, (1, T, 2, 128), dtype), _draw(g, (1, T, 1, 128), dtype), _draw(g, (1, T, 1, 128), dtype)
    up = (torch.linspace(0.02, 6.0, T, device="cuda") ** 2)[None, :, None, None]
    k = (k * up).to(k.dtype)
    o = G.gdn_attn_prefill(q, k, v)
    _check_rows(o[0], q[0], _np(k[0]), _np(v[0]), 0, 128 ** -0.5, dtype, None, "growing", _some(T, 1))
    o = G.gdn_attn_prefill(q, k.flip(1).contiguous(), v)
    _check_rows(o[0], q[0], _np(k[0]).copy()[::-1], _np(v[0]), 0, 128 ** -0.5, dtype, None, "falling", _some(T, 2))


def test_prefill_narrow_heads_growing_and_sharp_scores():
    """The same at the other head width."""
    torch, G = _torch()
    g = _gen(13)
    T = 700
    q, k, v = _draw(g, (1, T, 2, 64), "bf16"), _draw(g, (1, T, 1, 64), "bf16"), _draw(g, (1, T, 1, 64), "bf16")
    up = (torch.linspace(0.02, 6.0, T, device="cuda") ** 2)[None, :, None, None]
    k = (k * up).to(k.dtype)
    o = G.gdn_attn_prefill(q, k, v)
    _check_rows(o[0], q[0], _np(k[0]), _np(v[0]), 0, 0.125, "bf16", None, "growing", _some(T, 1))
    o = G.gdn_attn_prefill(q, k.flip(1).contiguous(), v)
    _check_rows(o[0], q[0], _np(k[0]).copy()[::-1], _np(v[0]), 0, 0.125, "bf16", None, "falling", _some(T, 2))


JUMPS = [20, 100, 126, 127, 128, 129, 130, 150, 160, 200, 250, 260, 300, 390, 450, 511, 520, 2000]


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_one_key_far_above_the_others(D):
    """One key whose score is `jump` (in powers of two of its weight) above all others, in a step that the
    rows see whole and after one that has set their reference, at every place modulo 16."""
    torch, G = _torch()
    g = _gen(18)
    T, cases = 384, [(j, p) for j in JUMPS for p in range(16)]
    q = torch.full((1, T * len(cases), 1, D), 8.0, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(q), _draw(g, q.shape, "bf16")
    for i, (jump, place) in enumerate(cases):           # scale q . k = k, with q = 8 and scale 1 / (8 D)
        k[0, i * T + 128 + 48 + place] = jump * np.log(2.0)
    o = G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32(_cu([T] * len(cases))), scale=1 / (8 * D))
    for i, (jump, place) in enumerate(cases):
        s = slice(i * T, i * T + T)
        _check_rows(o[0, s], q[0, s], _np(k[0, s]), _np(v[0, s]), 0, 1 / (8 * D), "bf16", None,
                    f"jump {jump} at {place}", [150, 256, 383])
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_paged_one_key_far_above_the_others(D):
    """The same where blocks share a tile's steps: in two steps one after the other, so that one of them is
    not the first of its block's."""
    torch, G = _torch()
    new, total = 20, 2000
    c = Cache([total], 1, D, 16, "bf16", 19)
    q = torch.full((new, 1, D), 8.0, dtype=torch.bfloat16, device="cuda")
    at = c.slots(0, 0, total)
    for jump in JUMPS:
        for place in (3, 14, 15):
            c.k.view(-1, 1, D)[at] = 0.0
            c.k.view(-1, 1, D)[at[[5 * 128 + 32 + place, 6 * 128 + 64 + place]]] = jump * np.log(2.0)
            o = G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32([0, new]), scale=1 / (8 * D))
            kn, vn = c.seq(0)
            _check_rows(o, q, kn, vn, total - new, 1 / (8 * D), "bf16", None, f"jump {jump} at {place}", [0, 19])
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_prefill_narrow_heads_other_scales(scale):
    torch, G = _torch()
    g = _gen(14)
    q, k, v = _draw(g, (1, 300, 2, 64), "bf16"), _draw(g, (1, 300, 2, 64), "bf16"), _draw(g, (1, 300, 2, 64), "bf16")
    o = G.gdn_attn_prefill(q, k, v, scale=scale)
    _check_rows(o[0], q[0], _np(k[0]), _np(v[0]), 0, scale, "bf16", None, f"scale {scale}", _some(300, 1, 8))


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_prefill_other_scales(scale):
    torch, G = _torch()
    g = _gen(14)
    q, k, v = _draw(g, (1, 140, 2, 128), "bf16"), _draw(g, (1, 140, 2, 128), "bf16"), _draw(g, (1, 140, 2, 128), "bf16")
    o = G.gdn_attn_prefill(q, k, v, scale=scale)
    _check_rows(o[0], q[0], _np(k[0]), _np(v[0]), 0, scale, "bf16", None, f"scale {scale}", _some(140, 1, 8))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prefill_nonfinite_in_masked_places(dtype, bad):
    """Keys and values that a row does not see may hold anything: the padding of a dense batch,
    the next sequence of a packed one, the row's own future."""
    torch, G = _torch()
    g = _gen(15)
    T, at = 400, 290
    q, k, v = _draw(g, (1, T, 4, 128), dtype), _draw(g, (1, T, 2, 128), dtype), _draw(g, (1, T, 2, 128), dtype)
    clean = G.gdn_attn_prefill(q, k, v)
    k2, v2 = k.clone(), v.clone()
    k2[:, at:], v2[:, at:] = bad, bad
    o = G.gdn_attn_prefill(q, k2, v2)
    _check_rows(o[0, :at], q[0, :at], _np(k[0]), _np(v[0]), 0, 128 ** -0.5, dtype, None, "before", _some(at, 1))
    far = at // 128 * 128 - 128                       # rows that share no tile with them: bit for bit
    assert torch.equal(o[:, :far], clean[:, :far])
    o = G.gdn_attn_prefill(q, k2, v2, cu_seqlens=_i32([0, at, T]))
    _check_rows(o[0, :at], q[0, :at], _np(k[0]), _np(v[0]), 0, 128 ** -0.5, dtype, None, "packed before", _some(at, 2))
    # and rows that do see a value that is not finite say so
    v3 = v.clone()
    v3[0, 100, 0, 5] = bad
    o = _np(G.gdn_attn_prefill(q, k, v3))
    assert np.isfinite(o[0, :100]).all() and np.isfinite(o[0, :, 2:]).all()
    assert not np.isfinite(o[0, 100:, :2, 5]).any() and np.isfinite(np.delete(o[0], 5, axis=2)).all()
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prefill_narrow_heads_nonfinite_in_masked_places(bad):
    """The rows' own future and the next sequence, at the other head width, with the edge at every place
    modulo 16."""
    torch, G = _torch()
    g = _gen(15)
    T = 400
    q, k, v = _draw(g, (1, T, 4, 64), "bf16"), _draw(g, (1, T, 2, 64), "bf16"), _draw(g, (1, T, 2, 64), "bf16")
    clean = G.gdn_attn_prefill(q, k, v)
    for at in range(280, 296):
        k2, v2 = k.clone(), v.clone()
        k2[:, at:], v2[:, at:] = bad, bad
        for cu in (None, _i32([0, at, T])):
            o = G.gdn_attn_prefill(q, k2, v2, cu_seqlens=cu)
            _check_rows(o[0, :at], q[0, :at], _np(k[0]), _np(v[0]), 0, 0.125, "bf16", None, f"before {at}", [0, 255, 256, at - 1])
            assert torch.equal(o[:, :128], clean[:, :128])
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prefill_nonfinite_keys_in_sight(dtype, bad, D):
    """A key that is not finite, its value finite, at every place modulo 16 of a step that the later rows
    see whole: NaN scores and scores of +inf make the rows that see them NaN, scores of -inf weigh nothing,
    and the rows before are as if it were not there."""
    torch, G = _torch()
    g = _gen(20)
    T, places, el = 400, range(16), 7
    n = len(places)
    q, k, v = (_draw(g, (1, T * n, h, D), dtype) for h in (2, 1, 1))
    q[0, :, 0, el] = q[0, :, 0, el].abs() + 0.25        # head 0's score has the sign of `bad`,
    q[0, :, 1, el] = -q[0, :, 1, el].abs() - 0.25       # head 1's the other
    clean = k.clone()
    at = [128 + 32 + p for p in places]
    for i, a in enumerate(at):
        k[0, i * T + a, 0, el] = bad
    o = G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32(_cu([T] * n)))
    for i, a in enumerate(at):
        s = slice(i * T, i * T + T)
        kn, vn, oi = _np(clean[0, s]), _np(v[0, s]), o[0, s]
        _check_rows(oi, q[0, s], kn, vn, 0, D ** -0.5, dtype, None, f"place {i}, before", [0, 127, 128, a - 1])
        for h in (0, 1):
            if np.isnan(bad) or (bad > 0) == (h == 0):
                assert torch.isnan(oi[a:, h]).all(), f"place {i} head {h}"
            else:
                _check_rows(oi[1:, h:h + 1], q[0, s][1:, h:h + 1], np.delete(kn, a, 0), np.delete(vn, a, 0), 0, D ** -0.5,
                            dtype, None, f"place {i} head {h}, behind", [a, 254, 255, 300, 382, 398])
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("D,HQ,HKV", [(128, 8, 2), (128, 4, 4), (64, 8, 2), (128, 6, 2)])
def test_prefill_back_to_back(D, HQ, HKV):
    """Many launches with no gap between them, over lengths at which a block's two tiles take
    different numbers of key steps: every one the same bits, no wait that runs out."""
    torch, G = _torch()
    g = _gen(16)
    lens = [2100, 130, 70, 1, 900, 257, 33, 1500]
    T, cu = sum(lens), _cu(lens)
    q, k, v = _draw(g, (1, T, HQ, D), "bf16"), _draw(g, (1, T, HKV, D), "bf16"), _draw(g, (1, T, HKV, D), "bf16")
    cud = _i32(cu)
    outs = [torch.empty_like(q) for _ in range(60)]
    ws = torch.empty(G.attn_prefill_workspace_bytes(T, len(lens), HQ, HKV, D, 1), dtype=torch.uint8, device="cuda")
    for o in outs:
        G.gdn_attn_prefill(q, k, v, cu_seqlens=cud, o=o, workspace=ws)
    assert G.gdn_attn_status() == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, outs[0]), i
    kn, vn = _np(k[0]), _np(v[0])
    for i in (0, 5):
        a, b = cu[i], cu[i + 1]
        _check_rows(outs[-1][0, a:b], q[0, a:b], kn[a:b], vn[a:b], 0, D ** -0.5, "bf16", None, f"sequence {i}",
                    _some(lens[i], i, 10))
    for _ in range(4000):
        G.gdn_attn_prefill(q, k, v, cu_seqlens=cud, o=outs[1], workspace=ws)
    assert G.gdn_attn_status() == 0 and torch.equal(outs[1], outs[0])


def test_paged_back_to_back_split():
    """The same for a few rows over long pasts, whose key ranges are shared between blocks."""
    torch, G = _torch()
    g = _gen(17)
    new, past = [20, 3, 1, 64, 33, 40], [7000, 130, 12000, 2500, 9001, 3000]
    totals = [n + p for n, p in zip(new, past)]
    c = Cache(totals, 8, 128, 16, "bf16", 18)
    q = _draw(g, (sum(new), 32, 128), "bf16")
    z = _draw(g, q.shape, "bf16")
    cud = _i32(_cu(new))
    ws = torch.empty(G.attn_prefill_workspace_bytes(sum(new), len(new), 32, 8, 128, 1), dtype=torch.uint8, device="cuda")
    call = lambda o: G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, cud, z=z, o=o, workspace=ws)
    outs = [call(torch.empty_like(q)) for _ in range(200)]
    o = torch.empty_like(q)
    for gated in (z, None):             # thousands of launches: a wait that is rarely missed shows
        for _ in range(4000):
            G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, cud, z=gated, o=o, workspace=ws)
        assert G.gdn_attn_status() == 0
    for i, x in enumerate(outs):
        assert torch.equal(x, outs[0]), i
    for i, n in enumerate(new):
        kn, vn = c.seq(i)
        a = _cu(new)[i]
        _check_rows(outs[0][a:a + n], q[a:a + n], kn, vn, past[i], 128 ** -0.5, "bf16", z[a:a + n], f"sequence {i}",
                    sorted({0, n // 2, n - 1}))


# ---- prompt pieces over the cache -----------------------------------------------------
PAGED = [
    # dtype, D, HQ, HKV, page, new, past, gate
    ("bf16", 128, 4, 2, 16, [1, 7, 0, 128], [0, 100, 50, 15], True),
    ("bf16", 128, 8, 1, 64, [130, 1], [129, 600], False),
    ("bf16", 128, 4, 4, 128, [257], [383], True),
    ("bf16", 64, 6, 2, 32, [33, 64, 5], [31, 0, 1000], False),
    ("bf16", 128, 2, 2, 16, [40, 3], [-25, -3], False),
    ("bf16", 128, 16, 2, 16, [3, 2, 9, 1], [2500, 1, 130, 4000], True),
    ("bf16", 64, 16, 4, 128, [600], [1500], False),
    ("fp32", 128, 4, 2, 16, [1, 70, 0], [64, 10, 3], True),
    ("fp32", 64, 5, 1, 128, [40, 3], [-25, 200], False),
]


@pytest.mark.parametrize("dtype,D,HQ,HKV,page,new,past,gate", PAGED)
def test_prefill_paged(dtype, D, HQ, HKV, page, new, past, gate):
    torch, G = _torch()
    g = _gen(21)
    totals = [n + p for n, p in zip(new, past)]
    c = Cache(totals, HKV, D, page, dtype, 22)
    T, cu = sum(new), _cu(new)
    q = _draw(g, (T + 3, HQ, D), dtype, 1.5)
    z = _draw(g, (T + 3, HQ, D), dtype) if gate else None
    o = torch.full_like(q, 7.0)
    G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32(cu), z=z, o=o)
    for i, n in enumerate(new):
        kn, vn = c.seq(i)
        a, b = cu[i], cu[i + 1]
        _check_rows(o[a:b], q[a:b], kn, vn, past[i], D ** -0.5, dtype, None if z is None else z[a:b],
                    f"sequence {i}", _some(n, i, 10))
    assert (o[T:] == 7.0).all()
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("new,past,page", [([130], [129], 16), ([3, 1], [130, 12000], 16), ([20, 64], [7000, 2500], 128),
                                           ([33, 257], [9001, 0], 64)])
def test_slots_past_the_contexts_cost_nothing(new, past, page):
    """Slots that no sequence holds (NaN here) are cleared on the way, not found in the outputs: the
    list of rows to do again (its length is word 1 of the workspace) stays empty."""
    torch, G = _torch()
    g = _gen(24)
    for D in (64, 128):
        c = Cache([n + p for n, p in zip(new, past)], 2, D, page, "bf16", 25)
        q = _draw(g, (sum(new), 8, D), "bf16")
        ws = torch.zeros(G.attn_prefill_workspace_bytes(sum(new), len(new), 8, 2, D, 1), dtype=torch.uint8, device="cuda")
        o = G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32(_cu(new)), workspace=ws)
        assert torch.isfinite(o).all() and ws[4:8].view(torch.int32).item() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("count,past0,page", [(400, 0, 16), (6, 5000, 64)])
def test_slots_past_the_contexts_where_both_tiles_end(D, count, past0, page):
    """Pieces of 64 tokens whose two tiles of 32 end in one step of 128 keys, as whole tiles and as tiles
    that blocks share: neither tile's product sees the slots behind the context (NaN here) before they
    are cleared, so no row is done again and every call gives the same bits."""
    torch, G = _torch()
    g = _gen(26)
    past = [past0 + 128 * (i % 3) + 13 * i % 64 for i in range(count)]
    assert all((p + 31) // 128 == (p + 63) // 128 for p in past)
    c = Cache([64 + p for p in past], 2, D, page, "bf16", 27)
    cu = _cu([64] * count)
    q = _draw(g, (cu[-1], 8, D), "bf16")
    ws = torch.zeros(G.attn_prefill_workspace_bytes(cu[-1], count, 8, 2, D, 1), dtype=torch.uint8, device="cuda")
    call = lambda o: G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32(cu), o=o, workspace=ws)
    first, o = call(torch.empty_like(q)), torch.empty_like(q)
    for _ in range(50):
        call(o)
        assert ws[4:8].view(torch.int32).item() == 0 and torch.equal(o, first)
    for i in (0, 1, count - 1):
        kn, vn = c.seq(i)
        _check_rows(o[64 * i:64 * i + 64], q[64 * i:64 * i + 64], kn, vn, past[i], D ** -0.5, "bf16", None,
                    f"sequence {i}", [0, 31, 32, 63])
    assert G.gdn_attn_status() == 0


# Prompts on the CUDA cores whose tiles several blocks share: few tiles (up to four pieces, from three
# steps of 64 keys on), and more (two or three, from six steps on); bf16 takes them for wide groups.
SHARED = [
    # dtype, D, HQ, HKV, lens, gate
    ("fp32", 64, 4, 2, [129], True),
    ("fp32", 128, 4, 1, [700], False),
    ("fp32", 64, 8, 2, [256, 193, 128, 1], True),
    ("fp32", 128, 2, 2, [65, 0, 450], False),
    ("fp32", 64, 8, 8, [500, 400, 330], True),
    ("fp32", 64, 8, 2, [900, 320, 321, 384, 500, 37], False),
    ("bf16", 64, 130, 1, [200], True),
]


@pytest.mark.parametrize("dtype,D,HQ,HKV,lens,gate", SHARED)
def test_prefill_shared_tiles(dtype, D, HQ, HKV, lens, gate):
    torch, G = _torch()
    g = _gen(71)
    cu = _cu(lens)
    q = _draw(g, (1, cu[-1], HQ, D), dtype, 1.5)
    k, v = (_draw(g, (1, cu[-1], HKV, D), dtype) for _ in range(2))
    z = _draw(g, q.shape, dtype) if gate else None
    call = lambda: G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32(cu), z=z)
    o = call()
    for i, n in enumerate(lens):
        r = slice(cu[i], cu[i + 1])
        rows = sorted({j for j in (0, 1, 63, 64, 65, 127, 128, 191, 192, 193, n // 2, n - 2, n - 1) if 0 <= j < n})
        _check_rows(o[0, r], q[0, r], _np(k[0, r]), _np(v[0, r]), 0, D ** -0.5, dtype,
                    None if z is None else z[0, r], f"seq {i}", rows)
    assert torch.equal(o, call())                                      # bit for bit
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_shared_tiles_nonfinite_in_masked_places(bad):
    """A key and a value late in the past leave the tokens before them alone, in a shared tile too."""
    torch, G = _torch()
    q, k, v = (_draw(_gen(72 + i), (1, 400, 2, 64), "fp32") for i in range(3))
    clean = G.gdn_attn_prefill(q, k, v)
    k[0, 301, 0, 3], v[0, 301, 0, 7] = bad, bad
    o = G.gdn_attn_prefill(q, k, v)
    assert torch.equal(o[:, :301], clean[:, :301]) and torch.equal(o[:, :, 1], clean[:, :, 1])
    assert not torch.isfinite(o[0, 399, 0, 7])
    assert G.gdn_attn_status() == 0


# Short pieces: at most 16 (token, head) rows a sequence on average; some longer ones among them.
SHORT = [
    # D, HQ, HKV, page, new, past, gate
    (128, 8, 2, 16, [4] * 5, [0, 100, 2500, 63, 17], True),
    (128, 4, 4, 64, [1, 16, 3], [300, 9000, 0], False),
    (64, 8, 2, 32, [1] * 12 + [20], [5, 0, 64, 700, 127, 128, 129, 1, 2, 3, 4, 3000, 900], True),
    (64, 6, 2, 128, [5, 0, 2, 6, 4], [1000, 50, 0, 31, 12000], False),          # 15 and 18 rows
    (128, 16, 1, 16, [1, 1, 0, 1], [4000, 0, 10, 129], True),
    (128, 16, 2, 64, [1] * 9 + [9], [77, 0, 500, 31, 32, 33, 2000, 63, 64, 400], False),
    (128, 4, 2, 16, [3, 2, 7, 4, 8], [-3, -1, -7, 60, -3], True),                # rows before the context
    (128, 1, 1, 16, [16, 17, 1, 3], [250, 1000, 0, 6000], False),
]


@pytest.mark.parametrize("D,HQ,HKV,page,new,past,gate", SHORT)
def test_short_pieces(D, HQ, HKV, page, new, past, gate):
    torch, G = _torch()
    assert sum(new) * (HQ // HKV) <= 16 * len(new)
    g = _gen(61)
    c = Cache([max(n + p, 0) for n, p in zip(new, past)], HKV, D, page, "bf16", 62)
    cu = _cu(new)
    q = _draw(g, (cu[-1], HQ, D), "bf16", 1.5)
    z = _draw(g, (cu[-1], HQ, D), "bf16") if gate else None
    ws = torch.zeros(G.attn_prefill_workspace_bytes(cu[-1], len(new), HQ, HKV, D, 1), dtype=torch.uint8, device="cuda")
    call = lambda: G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32(cu), z=z, workspace=ws)
    o = call()
    assert ws[4:8].view(torch.int32).item() == 0                       # no row done again
    for i, n in enumerate(new):
        if n == 0:
            continue
        kn, vn = c.seq(i) if c.totals[i] else (np.zeros((0, HKV, D)),) * 2
        r = slice(cu[i], cu[i + 1])
        _check_rows(o[r], q[r], kn, vn, c.totals[i] - n, D ** -0.5, "bf16", None if z is None else z[r], f"seq {i}")
    assert torch.equal(o, call())                                      # bit for bit
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("past", [37, 9000])
def test_short_pieces_nonfinite_in_masked_places(bad, past):
    """A value (or key) that only the later tokens of a piece see leaves the earlier ones alone, in a
    piece that one block holds and in one that many share."""
    torch, G = _torch()
    D, HQ, HKV, n = 128, 8, 2, 4
    g = _gen(63)
    for in_v in (True, False):
        c = Cache([past + n, past + n], HKV, D, 16, "bf16", 64)
        q = _draw(g, (2 * n, HQ, D), "bf16", 1.5)
        cu = _i32([0, n, 2 * n])
        clean = G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, cu)
        pos = past + 2                                                 # tokens 2 and 3 of the piece see it
        page = c.table[1, pos // 16].item()
        (c.v if in_v else c.k)[page, pos % 16, 1, 5] = bad
        o = G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, cu)
        assert torch.equal(o[:n], clean[:n])                           # another sequence
        assert torch.equal(o[n:, :4], clean[n:, :4])                   # the other key-value head
        kn, vn = c.seq(1)
        m = past + 2
        _check_rows(o[n:n + 2, 4:], q[n:n + 2, 4:], kn[:m, 1:], vn[:m, 1:], past, D ** -0.5, "bf16", None, "rows before")
        if in_v:
            assert not torch.isfinite(o[n + 2:, 4:, 5]).any()
        assert G.gdn_attn_status() == 0


def test_short_pieces_agree_with_decode():
    """Single tokens through the piece call are what the decode call returns, up to their roundings:
    each lies within the bound of the definition."""
    torch, G = _torch()
    r = np.random.default_rng(9)
    ctx = r.integers(1, 90, 700).tolist()
    ctx[300] = 5000
    c = Cache(ctx, 2, 64, 16, "bf16", 65)
    q = _draw(_gen(66), (len(ctx), 8, 64), "bf16", 1.5)
    o = G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32(list(range(len(ctx) + 1))))
    _check_decode(c, q, o, "bf16", None, 64 ** -0.5)
    _check_decode(c, q, G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens), "bf16", None, 64 ** -0.5)
    assert G.gdn_attn_status() == 0


def test_short_pieces_back_to_back():
    """Launches over one workspace, without a synchronisation between them, repeat bit for bit."""
    torch, G = _torch()
    new = [4] * 9 + [12]
    c = Cache([n + p for n, p in zip(new, [3000, 10, 777, 64, 1500, 0, 9000, 5, 128, 2000])], 4, 128, 16, "bf16", 67)
    cu = _i32(_cu(new))
    q = _draw(_gen(68), (sum(new), 12, 128), "bf16")
    ws = torch.empty(G.attn_prefill_workspace_bytes(sum(new), len(new), 12, 4, 128, 1), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    for i in range(600):
        G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, cu, o=outs[i > 0], workspace=ws)
    assert torch.equal(*outs)
    assert G.gdn_attn_status() == 0


# ---- decode -----------------------------------------------------------------------------
DECODE = [
    # dtype, D, HQ, HKV, page, contexts, gate
    ("bf16", 128, 4, 2, 16, [1, 0, 15, 16, 17, 63, 64, 65, 200], True),
    ("bf16", 128, 8, 1, 64, [5000], False),
    ("bf16", 128, 16, 1, 32, [129, 1, 700], True),
    ("bf16", 128, 20, 1, 16, [300, 31], False),
    ("bf16", 128, 7, 7, 128, [127, 128, 129], False),
    ("bf16", 64, 6, 2, 16, [1, 2, 3, 0, 1000], True),
    ("bf16", 64, 48, 1, 64, [333], False),
    ("bf16", 128, 32, 8, 64, [900, 12, 4000, 77], True),
    ("bf16", 128, 4, 1, 16, [20000], False),
    ("fp32", 128, 4, 2, 16, [1, 0, 33, 300], True),
    ("fp32", 64, 16, 16, 32, [65, 2, 700], False),
    ("fp32", 64, 10, 1, 128, [2000], True),
    ("fp32", 128, 40, 2, 64, [257, 9], False),
]


def _check_decode(c, q, o, dtype, z, scale, what=""):
    for i in range(q.shape[0]):
        kn, vn = c.seq(i) if c.totals[i] else (np.zeros((0,) + tuple(c.k.shape[2:])),) * 2
        want, bound = R.attention(_np(q[i:i + 1]), kn, vn, c.totals[i] - 1, scale, dtype,
                                  None if z is None else _np(z[i:i + 1]))
        _close(o[i:i + 1], want, bound, f"{what} sequence {i}")


@pytest.mark.parametrize("dtype,D,HQ,HKV,page,ctx,gate", DECODE)
def test_decode(dtype, D, HQ, HKV, page, ctx, gate):
    torch, G = _torch()
    g = _gen(31)
    c = Cache(ctx, HKV, D, page, dtype, 32)
    q = _draw(g, (len(ctx), HQ, D), dtype, 1.5)
    z = _draw(g, (len(ctx), HQ, D), dtype) if gate else None
    o = G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens, z=z)
    _check_decode(c, q, o, dtype, z, D ** -0.5)
    assert torch.equal(o, G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens, z=z))     # bit for bit
    assert G.gdn_attn_status() == 0


def test_decode_many_sequences():
    """More sequences than one pass of a block over the lengths, most of them short."""
    torch, G = _torch()
    g = _gen(33)
    r = np.random.default_rng(3)
    ctx = r.integers(0, 40, 1500).tolist()
    ctx[700] = 3000
    c = Cache(ctx, 1, 64, 16, "bf16", 34)
    q = _draw(g, (len(ctx), 2, 64), "bf16")
    o = G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens)
    _check_decode(c, q, o, "bf16", None, 64 ** -0.5)


def test_decode_growing_scores():
    torch, G = _torch()
    g = _gen(35)
    c = Cache([3001, 640], 1, 128, 64, "bf16", 36)
    for i, t in enumerate(c.totals):
        s = c.slots(i, 0, t)
        up = torch.linspace(0.02, 5.0, t, device="cuda")[:, None, None] ** 2
        c.k.view(-1, 1, 128)[s] = (c.k.view(-1, 1, 128)[s].float() * up).to(torch.bfloat16)
    q = _draw(g, (2, 4, 128), "bf16")
    _check_decode(c, q, G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens), "bf16", None, 128 ** -0.5)


def test_long_cache_offsets():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32)."""
    torch, G = _torch()
    g = _gen(37)
    page, HKV, D = 128, 8, 128
    n_pages = (1 << 31) // (page * HKV * D) + 40
    kc = torch.empty((n_pages, page, HKV, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    total, new = 300, 140
    table = _i32([[n_pages - 1, n_pages - 3, n_pages - 2]])
    k, v, q = (_draw(g, (total, h, D), "bf16") for h in (HKV, HKV, 16))
    lens = lambda n: _i32([n])
    G.gdn_attn_append(None, k, v, kc, vc, table, lens(total), cu_seqlens=_i32([0, total]))
    o = G.gdn_attn_decode(q[-1:].contiguous(), kc, vc, table, lens(total))
    _check_rows(o, q[-1:], _np(k), _np(v), total - 1, D ** -0.5, "bf16", None, "decode")
    o = G.gdn_attn_prefill_paged(q[-new:].contiguous(), kc, vc, table, lens(total), _i32([0, new]))
    _check_rows(o, q[-new:], _np(k), _np(v), total - new, D ** -0.5, "bf16", None, "paged", [0, 1, 77, new - 1])
    assert G.gdn_attn_status() == 0


# ---- wide groups, many sequences, gates at their ends -----------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("HQ,HKV", [(100, 1), (130, 1), (258, 2)])
def test_wide_groups(dtype, HQ, HKV):
    """Groups that leave a tile one token, and that no tile holds."""
    torch, G = _torch()
    g = _gen(61)
    lens = [9, 1, 40]
    T = sum(lens)
    q, k, v = _draw(g, (1, T, HQ, 64), dtype), _draw(g, (1, T, HKV, 64), dtype), _draw(g, (1, T, HKV, 64), dtype)
    z = _draw(g, q.shape, dtype)
    o = G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32(_cu(lens)), z=z)
    c = Cache([700, 3], HKV, 64, 16, dtype, 62)
    qd = _draw(g, (2, HQ, 64), dtype)
    od = G.gdn_attn_decode(qd, c.k, c.v, c.table, c.lens)
    kn, vn = _np(k[0]), _np(v[0])
    for i, n in enumerate(lens):
        a, b = _cu(lens)[i], _cu(lens)[i + 1]
        _check_rows(o[0, a:b], q[0, a:b], kn[a:b], vn[a:b], 0, 0.125, dtype, z[0, a:b], f"sequence {i}",
                    sorted({0, n // 2, n - 1}))
    _check_decode(c, qd, od, dtype, None, 0.125)
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_short_sequences(dtype):
    """More sequences than a plan block has threads, most of them of a few tokens, some empty."""
    torch, G = _torch()
    g = _gen(63)
    r = np.random.default_rng(5)
    new = r.integers(0, 9, 1500).tolist()
    new[1000] = 300
    past = r.integers(0, 40, 1500).tolist()
    totals = [n + p for n, p in zip(new, past)]
    c = Cache(totals, 1, 64, 16, dtype, 64)
    T, cu = sum(new), _cu(new)
    q, k, v = _draw(g, (T, 2, 64), dtype), _draw(g, (T, 1, 64), dtype), _draw(g, (T, 1, 64), dtype)
    qo = G.gdn_attn_append(q, k, v, c.k, c.v, c.table, c.lens, cu_seqlens=_i32(cu))
    assert torch.equal(qo, q)                                # no rotation
    o = G.gdn_attn_prefill_paged(qo, c.k, c.v, c.table, c.lens, _i32(cu))
    whole = G.gdn_attn_prefill(q[None], k[None], v[None], cu_seqlens=_i32(cu))[0]
    kn, vn = _np(k), _np(v)
    for i in [0, 1, 2, 999, 1000, 1001, 1023, 1024, 1025, 1499, *r.integers(0, 1500, 40).tolist()]:
        a, b = cu[i], cu[i + 1]
        rows = sorted({0, new[i] // 2, new[i] - 1}) if new[i] else []
        kc, vc = c.seq(i) if totals[i] else (None, None)
        _check_rows(o[a:b], q[a:b], kc, vc, past[i], 0.125, dtype, None, f"paged {i}", rows)
        _check_rows(whole[a:b], q[a:b], kn[a:b], vn[a:b], 0, 0.125, dtype, None, f"whole {i}", rows)
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gate_at_its_ends(dtype):
    """Gates of infinities are 0 and 1, very negative ones 0; a NaN gate is a NaN there only."""
    torch, G = _torch()
    g = _gen(65)
    c = Cache([500], 1, 128, 64, dtype, 66)
    for n in (1, 130):
        q = _draw(g, (n, 2, 128), dtype)
        cu, lens = _i32([0, n]), c.lens
        plain = _np(G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, lens, cu))
        z = torch.zeros_like(q)
        z[..., 0], z[..., 1], z[..., 2], z[..., 3], z[..., 4] = float("inf"), -float("inf"), -300.0, 300.0, float("nan")
        outs = [G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, lens, cu, z=z)]
        if n == 1:
            outs.append(G.gdn_attn_decode(q, c.k, c.v, c.table, lens, z=z))
        for o in outs:
            o = _np(o)
            assert np.isnan(o[..., 4]).all() and np.isfinite(np.delete(o, 4, axis=-1)).all()
            assert not o[..., 1].any() and not o[..., 2].any()
            tol = 3 * R.HALF_STEP[dtype] + 64 * R.U             # both sides rounded, and their sums' order
            for col, f in ((0, 1.0), (3, 1.0), (5, 0.5)):
                assert (np.abs(o[..., col] - f * plain[..., col]) <= tol * (np.abs(plain[..., col]) + 0.2)).all()
    assert G.gdn_attn_status() == 0


def test_two_graphs_share_a_workspace():
    """Two captured graphs over one workspace, replayed in turn on one stream."""
    torch, G = _torch()
    g = _gen(67)
    new, past = [33, 5], [5000, 77]
    totals = [n + p for n, p in zip(new, past)]
    c = Cache(totals, 2, 128, 64, "bf16", 68)
    T, cu = sum(new), _i32(_cu(new))
    q = [_draw(g, (T, 8, 128), "bf16") for _ in range(2)]
    qd = [_draw(g, (2, 8, 128), "bf16") for _ in range(2)]
    n = max(G.attn_prefill_workspace_bytes(T, 2, 8, 2, 128, 1), G.attn_decode_workspace_bytes(2, 8, 2, 128, 1))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    step = lambda i: (G.gdn_attn_prefill_paged(q[i], c.k, c.v, c.table, c.lens, cu, workspace=ws),
                      G.gdn_attn_decode(qd[i], c.k, c.v, c.table, c.lens, workspace=ws))
    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(step(i))
        graphs.append(graph)
    ws.fill_(255)                                            # what a workspace holds does not matter
    for _ in range(3):
        for i in (0, 1, 1, 0):
            for o in got[i]:
                o.zero_()
            graphs[i].replay()
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert G.gdn_attn_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new,total", [(0, 17), (0, 3000), (1, 17), (4, 3000), (20, 2000), (200, 200)])
def test_values_in_sight_behind_scores_of_minus_infinity(dtype, new, total):
    """A key whose score is -inf weighs nothing, and 0 * inf is NaN: an infinite value there makes its column
    NaN, whichever warp or block has only such keys (0 new tokens: decode).  The other columns are as if
    the keys were not there."""
    torch, G = _torch()
    g = _gen(69)
    D, col = 64, 5
    for a, b in ((16, 17), (64, 128), (512, 1536), (600, 601)):
        if b > total:
            continue
        c = Cache([total], 1, D, 16, dtype, 70)
        q = _draw(g, (max(new, 1), 2, D), dtype)
        q[..., 9] = q[..., 9].abs() + 0.25
        kn, vn = c.seq(0)
        at = c.slots(0, a, b)
        c.k.view(-1, 1, D)[at, :, 9] = -float("inf")
        c.v.view(-1, 1, D)[at, :, col] = float("inf")
        past = total - q.shape[0]
        rows = sorted({0, 15, 16, 17, 127, 128, 150, new // 2, new - 1} & set(range(q.shape[0]))) if new else [0]
        if new == 0:
            o = G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens)
        else:
            o = G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32([0, new]))
        for r in rows:
            seen = np.delete(np.arange(past + r + 1), np.arange(a, min(b, past + r + 1))) if past + r >= a else np.arange(past + r + 1)
            want, bound = R.attention(_np(q[r:r + 1]), kn[seen], vn[seen], len(seen) - 1, D ** -0.5, dtype)
            got = o[r:r + 1].clone()
            if past + r >= a:
                assert torch.isnan(got[..., col]).all(), (a, b, r)
                got[..., col] = torch.from_numpy(want[..., col]).to(got)
            _close(got, want, bound, f"keys {a} to {b}, row {r}")
    assert G.gdn_attn_status() == 0


def test_a_captured_call_with_other_lengths_and_pages():
    """A graph's calls read lengths and tables when they run: replayed as contexts grow, shrink and become
    idle, with another order of the pages and with pages that two sequences share."""
    torch, G = _torch()
    g = _gen(73)
    D, page = 128, 16
    longest = [1500, 700, 90, 3000]
    c = Cache(longest, 2, D, page, "bf16", 74)
    new = [20, 1, 3, 9]
    cu = _i32(_cu(new))
    q, qd = _draw(g, (sum(new), 8, D), "bf16"), _draw(g, (4, 8, D), "bf16")
    n = max(G.attn_prefill_workspace_bytes(sum(new), 4, 8, 2, D, 1), G.attn_decode_workspace_bytes(4, 8, 2, D, 1))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    step = lambda: (G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, cu, workspace=ws),
                    G.gdn_attn_decode(qd, c.k, c.v, c.table, c.lens, workspace=ws))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op, od = step()
    for totals, rows in (([1500, 700, 90, 3000], [0, 1, 2, 3]), ([1, 0, 90, 17], [0, 1, 2, 3]),
                         ([700, 690, 90, 2999], [1, 1, 2, 3]), ([33, 64, 65, 1024], [3, 0, 1, 3])):
        c.totals = totals
        c.lens.copy_(_i32(totals))
        keep = c.table_np
        c.table_np = keep[rows]
        c.table.copy_(torch.from_numpy(c.table_np))
        graph.replay()
        _check_decode(c, qd, od, "bf16", None, D ** -0.5, f"lengths {totals}")
        for i, n in enumerate(new):
            kn, vn = c.seq(i) if totals[i] else (np.zeros((0, 2, D)),) * 2
            r = slice(_cu(new)[i], _cu(new)[i + 1])
            _check_rows(op[r], q[r], kn, vn, totals[i] - n, D ** -0.5, "bf16", None, f"lengths {totals}, sequence {i}")
        c.table_np = keep
    assert G.gdn_attn_status() == 0


# ---- bad tables (checked by paged.cuh, whose arithmetic test_attn_ref.py checks) --------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_bad_tables_are_reported_and_stay_contained(dtype):
    torch, G = _torch()
    g = _gen(41)
    c = Cache([40, 300, 100], 2, 128, 16, dtype, 42)
    q = _draw(g, (3, 4, 128), dtype)
    good = G.gdn_attn_decode(q, c.k, c.v, c.table, c.lens)
    for value in (-7, c.k.shape[0], 2 ** 31 - 1):
        t = c.table.clone()
        t[1, 3] = value
        o = G.gdn_attn_decode(q, c.k, c.v, t, c.lens)
        assert G.gdn_attn_status() == 3 and G.gdn_attn_status() == 0
        assert torch.equal(o[[0, 2]], good[[0, 2]])
        cu = _i32([0, 1, 2, 3])
        p = G.gdn_attn_prefill_paged(q, c.k, c.v, t, c.lens, cu)
        assert G.gdn_attn_status() == 3
        _check_decode(c, q[:1], p[:1], dtype, None, 128 ** -0.5)
        # the third sequence's own row, against the reference
        kn, vn = c.seq(2)
        _check_rows(p[2:3], q[2:3], kn, vn, 99, 128 ** -0.5, dtype, None, "third")
    # a context longer than its table row, a negative one: the sequence is skipped
    for value in (c.table.shape[1] * 16 + 1, -1):
        lens = c.lens.clone()
        lens[1] = value
        o = torch.full_like(q, 7.0)
        G.gdn_attn_decode(q, c.k, c.v, c.table, lens, o=o)
        assert G.gdn_attn_status() == 3
        # (the lengths of a batch decide where its work is split, so the others' sums may be taken
        # in another order: the reference's bound, not the same bits)
        for i in (0, 2):
            kn, vn = c.seq(i)
            _check_rows(o[i:i + 1], q[i:i + 1], kn, vn, c.totals[i] - 1, 128 ** -0.5, dtype, None, f"sequence {i}")
        assert (o[1] == 7.0).all()
        k, v = _draw(g, (3, 2, 128), dtype), _draw(g, (3, 2, 128), dtype)
        kc, vc = c.k.clone(), c.v.clone()
        qo = torch.full_like(q, 7.0)
        G.gdn_attn_append(q, k, v, kc, vc, c.table, lens, q_out=qo)
        assert G.gdn_attn_status() == 3 and (qo[1] == 7.0).all()
        assert torch.isnan(kc).sum() == torch.isnan(c.k).sum()
    # sequences out of order
    for cu in ([0, 2, 1, 3], [0, 1, 2, 4], [1, 1, 2, 3]):
        o = torch.full_like(q, 7.0)
        G.gdn_attn_prefill_paged(q, c.k, c.v, c.table, c.lens, _i32(cu), o=o)
        assert G.gdn_attn_status() == 1, cu
        G.gdn_attn_append(q, _draw(g, (3, 2, 128), dtype), _draw(g, (3, 2, 128), dtype), c.k.clone(), c.v.clone(),
                          c.table, c.lens, cu_seqlens=_i32(cu), q_out=o)
        assert G.gdn_attn_status() == 1, cu
    # an append through a bad page writes nothing there
    t = c.table.clone()
    t[0, 39 // 16] = c.k.shape[0] + 5
    kc, vc = c.k.clone(), c.v.clone()
    G.gdn_attn_append(None, _draw(g, (3, 2, 128), dtype), _draw(g, (3, 2, 128), dtype), kc, vc, t, c.lens)
    assert G.gdn_attn_status() == 3
    s = c.slots(0, 0, 40)
    assert torch.equal(kc.view(-1, 256)[s], c.k.view(-1, 256)[s])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("count", [9, 199])
def test_sequences_that_name_the_same_rows_over_and_over(dtype, count):
    """A cu_seqlens that goes up and down gives many sequences all rows: more tiles than the plan has room for,
    however few or many.  None is listed, and the next call over the workspace is as ever."""
    torch, G = _torch()
    g = _gen(43)
    T, H = 1000, 8
    q, k, v = (_draw(g, (1, T, H, 64), dtype) for _ in range(3))
    ws = torch.empty(G.attn_prefill_workspace_bytes(T, count, H, H, 64, int(dtype == "bf16")), dtype=torch.uint8, device="cuda")
    o = torch.full_like(q, 7.0)
    G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32([T * (i & 1) for i in range(count + 1)]), o=o, workspace=ws)
    assert G.gdn_attn_status() == 1 and (o == 7.0).all()
    G.gdn_attn_prefill(q, k, v, cu_seqlens=_i32([0] * count + [T]), o=o, workspace=ws)
    _check_rows(o[0], q[0], _np(k[0]), _np(v[0]), 0, 0.125, dtype, None, "one sequence", [0, 500, T - 1])
    assert G.gdn_attn_status() == 0


# ---- as they are used -----------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_prompt_in_pieces_then_tokens_equals_the_whole(dtype):
    """append + prefill_paged over pieces, then append + decode token by token, against
    prefill of the whole and the reference."""
    torch, G = _torch()
    g = _gen(51)
    T, HQ, HKV, D, page = 330, 4, 2, 128, 16
    q, k, v = _draw(g, (T, HQ, D), dtype), _draw(g, (T, HKV, D), dtype), _draw(g, (T, HKV, D), dtype)
    z = _draw(g, (T, HQ, D), dtype)
    f = (1e4 ** -(torch.arange(0, 64, 2, device="cuda") / 64)).float()
    width = -(-T // page)
    table = torch.randperm(width + 4, generator=g, device="cuda")[:width].int()[None].contiguous()
    kc = torch.full((width + 4, page, HKV, D), float("nan"), dtype=q.dtype, device="cuda")
    vc = kc.clone()
    o, qr = torch.empty_like(q), torch.empty_like(q)
    at = 0
    for n in (200, 1, 100):
        sl = slice(at, at + n)
        cu, lens = _i32([0, n]), _i32([at + n])
        G.gdn_attn_append(q[sl], k[sl], v[sl], kc, vc, table, lens, cu_seqlens=cu, inv_freq=f, q_out=qr[sl])
        G.gdn_attn_prefill_paged(qr[sl], kc, vc, table, lens, cu, z=z[sl], o=o[sl])
        at += n
    while at < T:
        sl = slice(at, at + 1)
        lens = _i32([at + 1])
        G.gdn_attn_append(q[sl], k[sl], v[sl], kc, vc, table, lens, inv_freq=f, q_out=qr[sl])
        G.gdn_attn_decode(qr[sl], kc, vc, table, lens, z=z[sl], o=o[sl])
        at += 1
    slots = (table[0].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:T]
    kr = kc.view(-1, HKV, D)[slots].contiguous()
    whole = G.gdn_attn_prefill(qr[None], kr[None], v[None], z=z[None])[0]
    kn, vn = _np(kr), _np(v)
    _check_rows(o, qr, kn, vn, 0, D ** -0.5, dtype, z, "pieces", _some(T, 1))
    _check_rows(whole, qr, kn, vn, 0, D ** -0.5, dtype, z, "whole", _some(T, 2))
    assert G.gdn_attn_status() == 0


def test_attention_layer_beside_the_delta_rule_layer():
    """One step of the hybrid stack: the delta-rule call and the attention calls over one packed
    batch (one cu_seqlens), captured into a graph and replayed with new inputs."""
    torch, G = _torch()
    g = _gen(52)
    lens = [70, 129, 1]
    T, cu = sum(lens), _i32(_cu(lens))
    HQ, HKV, D, page = 4, 2, 128, 16
    c = Cache(lens, HKV, D, page, "bf16", 53)
    x = _draw(g, (T, (HQ + 2 * HKV) * D), "bf16")
    gd, beta = -torch.rand((1, T, HQ), device="cuda"), torch.rand((1, T, HQ), device="cuda")
    f = torch.rand(64, device="cuda")
    ws = torch.empty(G.attn_prefill_workspace_bytes(T, 3, HQ, HKV, D, 1), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(G.prefill_workspace_bytes(T, 3, HKV, HQ, D, D, 64, 1), dtype=torch.uint8, device="cuda")
    dws = torch.empty(G.attn_decode_workspace_bytes(3, HQ, HKV, D, 1), dtype=torch.uint8, device="cuda")
    qo, o, od = (torch.empty((T, HQ, D), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    last = torch.tensor(_cu(lens)[1:], device="cuda") - 1

    def step():
        q, k, v = (x[:, :HQ * D].unflatten(1, (HQ, D)), x[:, HQ * D:(HQ + HKV) * D].unflatten(1, (HKV, D)),
                   x[:, (HQ + HKV) * D:].unflatten(1, (HKV, D)))
        G.gdn_chunk_prefill(k.contiguous()[None], v.contiguous()[None], q.contiguous()[None], gd, beta, cu_seqlens=cu,
                            workspace=ws2)
        G.gdn_attn_append(q, k, v, c.k, c.v, c.table, c.lens, cu_seqlens=cu, inv_freq=f, q_out=qo)
        G.gdn_attn_prefill_paged(qo, c.k, c.v, c.table, c.lens, cu, o=o, workspace=ws)
        ql = qo[last].contiguous()
        return G.gdn_attn_decode(ql, c.k, c.v, c.table, c.lens, workspace=dws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        od = step()
    for seed in (1, 2):
        x.copy_(_draw(_gen(seed), x.shape, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        for i, n in enumerate(lens):
            kn, vn = c.seq(i)
            a, b = _cu(lens)[i], _cu(lens)[i + 1]
            _check_rows(o[a:b], qo[a:b], kn, vn, 0, D ** -0.5, "bf16", None, f"replay, sequence {i}", _some(n, i, 4))
            _check_rows(od[i:i + 1], qo[b - 1:b], kn, vn, n - 1, D ** -0.5, "bf16", None, f"replay, decode {i}")
    assert G.gdn_attn_status() == 0


def test_two_streams_at_once():
    torch, G = _torch()
    g = _gen(54)
    T = 600
    q, k, v = _draw(g, (2, 1, T, 4, 128), "bf16"), _draw(g, (2, 1, T, 2, 128), "bf16"), _draw(g, (2, 1, T, 2, 128), "bf16")
    c = Cache([3000, 17], 2, 128, 64, "bf16", 55)
    qd = _draw(g, (2, 4, 128), "bf16")
    want = [G.gdn_attn_prefill(q[i], k[i], v[i]) for i in range(2)]
    wd = G.gdn_attn_decode(qd, c.k, c.v, c.table, c.lens)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got, gd = [[], []], [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                got[i].append(G.gdn_attn_prefill(q[i], k[i], v[i]))
                gd[i].append(G.gdn_attn_decode(qd, c.k, c.v, c.table, c.lens))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i]) and all(torch.equal(x, wd) for x in gd[i])


def test_binding_refusals():
    torch, G = _torch()
    c = Cache([20], 2, 128, 16, "bf16", 1)
    q, k = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    tab = (c.k, c.v, c.table, c.lens)
    with pytest.raises(TypeError):
        G.gdn_attn_decode(q.float(), *tab)
    with pytest.raises(ValueError):
        G.gdn_attn_decode(torch.cat([q, q]), *tab)                    # a row more than the table
    with pytest.raises(TypeError):
        G.gdn_attn_decode(q, c.k, c.v, c.table.long(), c.lens)
    with pytest.raises(ValueError):
        G.gdn_attn_decode(q, c.k, c.v, c.table.cpu(), c.lens)
    with pytest.raises(ValueError):
        G.gdn_attn_decode(q.transpose(1, 2).contiguous().transpose(1, 2), *tab)      # not contiguous
    with pytest.raises(ValueError):
        G.gdn_attn_append(q, k, k[..., :64], *tab)
    with pytest.raises(ValueError):
        G.gdn_attn_append(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, *tab)      # heads strided
    with pytest.raises(TypeError):
        G.gdn_attn_append(q, k, k, *tab, inv_freq=torch.zeros(16, device="cuda", dtype=torch.float64))
    with pytest.raises(G.GDNError):
        G.gdn_attn_append(q, k, k, *tab, inv_freq=torch.zeros(12, device="cuda"))
    with pytest.raises(ValueError):
        G.gdn_attn_prefill(q[None], k[None], k[None, :, :1])
    with pytest.raises(ValueError):
        G.gdn_attn_prefill(q[None], k[None], k[None], z=q)
    with pytest.raises(G.GDNError):
        G.gdn_attn_prefill(q[None], k[None], k[None], o=q[None])       # o over q
    with pytest.raises(ValueError):
        G.gdn_attn_prefill_paged(q, *tab, _i32([0, 1, 1]))
