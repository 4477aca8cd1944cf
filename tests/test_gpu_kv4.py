"""csa_qk_norm_rope and the 4-bit cache on the GPU, against the plain float64
restatement in oracle/kv4.py.

Tolerances are derived, not fitted:
  * codes, bounds and scales: bit for bit; rows read back: the float32 value,
    rounded once to the type, bit for bit;
  * norms and rotation: the float32 chain has at most 12 roundings of half a
    step of 2^-24 that act on a term no larger than |x_a| + |x_b| (norm,
    weight, angle, sine or cosine to 2 ulp, products, sum), so 24 * 2^-24
    (|a| + |b|) covers it, plus half a step of the output type;
  * attention: a score's rounding error is at most eps_s = (2^-21 + 8 sqrt(d)
    2^-24) S, S = max over tokens of sum_c |q_c| (|m_c| + 15 Delta_c) /
    sqrt(d) (products to 22 bits, and d roundings of independent sign at
    eight standard deviations); it moves every weight by a factor within exp(+-eps_s),
    so the output by at most 2 eps_s vmax; the weights and sums over n tokens
    add (2^-20 + 8 sqrt(n) 2^-24) vmax, vmax the largest |v| stood for.
"""
import numpy as np
import pytest

from oracle import kv4
from oracle.quantize import quantize_keys
from tests.gpu_common import ensure_built

pytestmark = pytest.mark.gpu
BLOCK = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _t():
    import torch
    import certified_sparse_attention_gb300 as csa
    return torch, csa, torch.device("cuda:0")


def tdtype(dtype):
    torch = _t()[0]
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def i64(xs):
    torch, _, dev = _t()
    return torch.tensor([int(x) for x in xs], dtype=torch.int64, device=dev)


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(rng, size, dtype):
    """Random rows with a few strong channels, in the type."""
    torch, _, dev = _t()
    x = rng.normal(size=size).astype(np.float32)
    x[..., :3] *= 6
    return torch.from_numpy(x).to(dev).to(tdtype(dtype))


# ------------------------------------------------------- norms and rotation

def check_rope(got, x, w, pos, f, inter, eps, dtype):
    """got, x float64 [d] of one row."""
    ref = kv4.norm_rope(x, w, eps, pos, f, inter)
    y = kv4.norm_rope(x, w, eps, pos, [], inter)         # normed, not rotated
    mag = np.abs(y).copy()
    n = len(f)
    if n:
        ia = np.arange(n) * 2 if inter else np.arange(n)
        ib = ia + 1 if inter else ia + n
        mag[ia] = mag[ib] = np.abs(y[ia]) + np.abs(y[ib])
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    lim = 24 * 2.0 ** -24 * mag * (1 + half) + half * np.abs(ref) + 1e-37
    assert np.all(np.abs(got - ref) <= lim), np.max(np.abs(got - ref) / lim)


@pytest.mark.parametrize("dtype,d,rot,inter,normed,cache", [
    ("bf16", 128, 128, False, True, True), ("bf16", 128, 128, True, True, False),
    ("f32", 64, 32, False, True, True), ("f32", 64, 24, True, False, False),
    ("f32", 128, 8, False, True, True), ("bf16", 64, 0, False, True, False),
    ("bf16", 64, 64, False, False, True), ("f32", 128, 104, True, True, True)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 8), (5, 8, 1), (3, 12, 3)])
def test_norm_rope(dtype, d, rot, inter, normed, cache, T, Hq, Hkv):
    torch, csa, dev = _t()
    rng = np.random.default_rng(rot + T)
    B, n_max = 3, 40
    new = [T, max(0, T - 1), T]
    lens = [n_max, new[1] + 7, T]
    qkv = rows(rng, (B, T, Hq + 2 * Hkv, d), dtype)      # side by side
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    wq = rows(rng, (d,), dtype) if normed else None
    wk = rows(rng, (d,), dtype) if normed else None
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    s = csa.make_shape(B, Hq, Hkv, d, n_max, dtype)
    op = csa.QKNormRope(s, dev, wq, wk, 1e-5, f if rot else None, inter)
    size = (B, Hkv, n_max, d) if cache else (B, T, Hkv, d)
    K = torch.full(size, 7.0, dtype=tdtype(dtype), device=dev)
    V = torch.full_like(K, 9.0)
    qo = torch.full((B, T, Hq, d), 5.0, dtype=tdtype(dtype), device=dev)
    assert op(q, k, v, K, V, i64(lens), i64(new), to_cache=cache, q_out=qo) is qo
    assert csa.csa_check(op.status) == 0
    Kn, Vn, qn = f64(K), f64(V), f64(qo)
    x = f64(qkv)
    wqn, wkn = (f64(wq), f64(wk)) if normed else (None, None)
    wrote = np.zeros(size[:-1], bool)
    for b in range(B):
        for t in range(T):
            if t >= new[b]:
                assert np.all(qn[b, t] == 5.0)
                continue
            pos = lens[b] - new[b] + t
            for h in range(Hq):
                check_rope(qn[b, t, h], x[b, t, h], wqn, pos, f, inter, 1e-5, dtype)
            for g in range(Hkv):
                at = (b, g, pos) if cache else (b, t, g)
                wrote[at] = True
                check_rope(Kn[at], x[b, t, Hq + g], wkn, pos, f, inter, 1e-5, dtype)
                assert np.array_equal(Vn[at], x[b, t, Hq + Hkv + g])
    assert np.all(Kn[~wrote] == 7.0) and np.all(Vn[~wrote] == 9.0)


def test_rope_far_positions_and_without_values():
    # angles at positions up to 2^31 - 1, in place, V left alone
    torch, csa, dev = _t()
    rng = np.random.default_rng(2)
    B, T, H, d = 4, 3, 2, 64
    f = 500000.0 ** (-np.arange(32) / 32)
    s = csa.make_shape(B, H, H, d, 1 << 31, "f32")
    op = csa.QKNormRope(s, dev, inv_freq=f)
    q, k = rows(rng, (B, T, H, d), "f32"), rows(rng, (B, T, H, d), "f32")
    x = f64(q)
    lens = [(1 << 31), 1234567, 1 << 24, 3]
    ko = torch.zeros_like(k)
    out = op(q, k, None, ko, None, i64(lens), None, to_cache=False, q_out=q)
    assert out is q
    got = f64(q)
    kx, kg = f64(k), f64(ko)
    for b in range(B):
        for t in range(T):
            for h in range(H):
                pos = lens[b] - T + t
                check_rope(got[b, t, h], x[b, t, h], None, pos, f, False, 0, "f32")
                check_rope(kg[b, t, h], kx[b, t, h], None, pos, f, False, 0, "f32")


def test_rope_strided_operands_and_made_output():
    # heads-major q (a transposed view), broadcast batch axis of k
    torch, csa, dev = _t()
    rng = np.random.default_rng(4)
    B, T, Hq, Hkv, d = 2, 6, 4, 2, 128
    s = csa.make_shape(B, Hq, Hkv, d, 50, "bf16")
    f = 10000.0 ** (-np.arange(64) / 64)
    w = rows(rng, (d,), "bf16")
    op = csa.QKNormRope(s, dev, w, w, inv_freq=f, interleaved=True)
    q = rows(rng, (B, Hq, T, d), "bf16").transpose(1, 2)
    k = rows(rng, (1, T, Hkv, d), "bf16").expand(B, T, Hkv, d)
    K = torch.zeros(B, Hkv, 50, d, dtype=torch.bfloat16, device=dev)
    V = torch.zeros_like(K)
    out = op(q, k, k, K, V, i64([6, 50]))
    ref = op(q.contiguous(), k.contiguous(), k.contiguous(), K.clone(),
             V.clone(), i64([6, 50]))
    assert torch.equal(out, ref) and out.shape == (B, T, Hq, d)
    assert torch.equal(V[1, :, 44:], k[1].transpose(0, 1))


def test_rope_range_is_reported():
    torch, csa, dev = _t()
    s = csa.make_shape(3, 2, 2, 64, 20, "bf16")
    op = csa.QKNormRope(s, dev)
    x = torch.ones(3, 4, 2, 64, dtype=torch.bfloat16, device=dev)
    for lens, new in (([21, 20, 20], [4, 4, 4]), ([20, 3, 20], [4, 4, 4]),
                      ([20, 20, 20], [4, 5, 4]), ([20, 20, 20], [4, 4, -1])):
        K = torch.zeros(3, 2, 20, 64, dtype=torch.bfloat16, device=dev)
        V, qo = torch.zeros_like(K), torch.zeros_like(x)
        op(x, x, x, K, V, i64(lens), i64(new), q_out=qo)
        assert csa.csa_check(op.status) == 1
        for b in range(3):
            ok = 0 <= new[b] <= 4 and new[b] <= lens[b] <= 20
            assert bool((K[b] != 0).any()) == ok and bool((qo[b] != 0).any()) == ok
        op(x, x, x, K, V, i64([20, 20, 20]))
        assert csa.csa_check(op.status) == 0


# ------------------------------------------------------------ the cache

class Model:
    """Rows appended so far, and what the cache stands for."""

    def __init__(self, B, H, d):
        self.k = [[np.zeros((0, d), np.float32) for _ in range(H)] for _ in range(B)]
        self.v = [[np.zeros((0, d), np.float32) for _ in range(H)] for _ in range(B)]

    def add(self, k, v, new):
        """k, v float32 [B][T][H][d]."""
        for b, m in enumerate(new):
            for g in range(len(self.k[b])):
                self.k[b][g] = np.concatenate([self.k[b][g], k[b, :m, g]])
                self.v[b][g] = np.concatenate([self.v[b][g], v[b, :m, g]])

    def stands(self, b, g):
        """float32 rows K, V, and per-row magnitudes |m| + 15 Delta of K."""
        k, v = self.k[b][g].copy(), self.v[b][g].copy()
        mag = np.abs(k)
        w = len(k) // BLOCK * BLOCK
        if w:
            c, _, m, dl = quantize_keys(k[:w], w)
            m, dl = np.repeat(m, BLOCK, 0), np.repeat(dl, BLOCK, 0)
            k[:w] = kv4.stands_for(c, m, dl)
            mag[:w] = np.abs(m) + 15 * dl
            c, m, dl = kv4.quantize_values(v[:w])
            v[:w] = kv4.stands_for(c, m[:, None], dl[:, None])
        return k, v, mag


def float32(t):
    return t.detach().float().cpu().numpy()


def append(cache, model, rng, dtype, lens, new, T):
    """Append random rows; rows past new[b] are NaN."""
    B, H, d = len(lens), cache.shape.Hkv, cache.shape.d
    k, v = rows(rng, (B, T, H, d), dtype), rows(rng, (B, T, H, d), dtype)
    model.add(float32(k), float32(v), new)
    for b in range(B):
        k[b, new[b]:] = float("nan")
        v[b, new[b]:] = float("nan")
    lens = [a + b for a, b in zip(lens, new)]
    cache.append(k, v, i64(lens), i64(new))
    return lens


@pytest.mark.parametrize("dtype,d,H", [("bf16", 128, 2), ("f32", 64, 3),
                                       ("bf16", 64, 1), ("f32", 128, 1)])
def test_append_and_unpack_bit_for_bit(dtype, d, H):
    torch, csa, dev = _t()
    rng = np.random.default_rng(d + H)
    B, n_max = 3, 400
    s = csa.make_shape(B, H, H, d, n_max, dtype)
    cache = csa.KV4Cache(s, dev)
    for name, x in (("K4", 0xA5), ("V4", 0x5A)):
        getattr(cache, name).fill_(x)
    for name in ("bounds", "vscale", "Kt", "Vt"):
        getattr(cache, name).fill_(-77.0)
    model, lens = Model(B, H, d), [0] * B
    for new in ([1, 0, 64], [62, 63, 1], [1, 2, 0], [0, 0, 0], [65, 1, 127],
                [130, 61, 64], [7, 1, 130]):
        lens = append(cache, model, rng, dtype, lens, new, max(1, max(new)))
        assert csa.csa_check(cache.status) == 0
        K4 = cache.K4.cpu().numpy()
        V4 = cache.V4.cpu().numpy()
        bounds, vs = cache.bounds.cpu().numpy(), cache.vscale.cpu().numpy()
        Kt, Vt = float32(cache.Kt), float32(cache.Vt)
        for b in range(B):
            w = lens[b] // BLOCK * BLOCK
            for g in range(H):
                k, v = model.k[b][g], model.v[b][g]
                _, packed, m, dl = quantize_keys(k[:w], w)
                assert np.array_equal(K4[b, g, :w], packed)
                assert np.array_equal(bounds[b, g, :w // BLOCK, 0], m)
                assert np.array_equal(bounds[b, g, :w // BLOCK, 1], dl)
                c, m, dl = kv4.quantize_values(v[:w]) if w else (0, [], [])
                assert np.array_equal(vs[b, g, :w, 0], m)
                assert np.array_equal(vs[b, g, :w, 1], dl)
                for j in range(w // BLOCK):
                    assert np.array_equal(V4[b, g, j], kv4.pack_values(
                        c[j * BLOCK:(j + 1) * BLOCK]))
                r = lens[b] - w
                assert np.array_equal(Kt[b, g, :r], k[w:])
                assert np.array_equal(Vt[b, g, :r], v[w:])
                # nothing past the whole blocks is written
                assert np.all(K4[b, g, w:] == 0xA5) and np.all(V4[b, g, w // BLOCK:] == 0x5A)
                assert np.all(bounds[b, g, w // BLOCK:] == -77) and np.all(vs[b, g, w:] == -77)
        # read back, whole and in part; rows past the end stay as they were
        for first, count in ((None, n_max), ([0, 3, 70], 50), ([5, 0, 129], 1), ([63, 64, 65], 129)):
            K = torch.full((B, H, count, d), 3.0, dtype=tdtype(dtype), device=dev)
            V = torch.full_like(K, 4.0)
            cache.unpack(K, V, i64(lens), None if first is None else i64(first))
            assert csa.csa_check(cache.status) == 0
            for b in range(B):
                f = 0 if first is None else first[b]
                m = max(0, min(lens[b], f + count) - f)
                for g in range(H):
                    k, v, _ = model.stands(b, g)
                    for got, want, rest in ((K, k, 3.0), (V, v, 4.0)):
                        want = torch.from_numpy(want[f:f + m]).to(tdtype(dtype))
                        assert torch.equal(got[b, g, :m].cpu(), want)
                        assert bool((got[b, g, m:] == rest).all())


def test_append_matches_the_key_quantiser():
    # the keys' codes and bounds are csa_quantize_keys' own
    torch, csa, dev = _t()
    rng = np.random.default_rng(8)
    B, H, d, n = 2, 2, 128, 192
    s = csa.make_shape(B, H, H, d, n, "bf16")
    K = rows(rng, (B, H, n, d), "bf16")
    meta = csa.meta_buffers(s, dev)
    csa.check(csa.csa_quantize_keys(s, K, K, [n, n], 0, *meta))
    cache = csa.KV4Cache(s, dev)
    cache.append(K.transpose(1, 2), K.transpose(1, 2), i64([n, n]))
    assert torch.equal(cache.K4, meta.K4) and torch.equal(cache.bounds, meta.bounds)


def test_append_special_values():
    # constant rows and channels; a NaN or infinity spoils its key channel of
    # the block and its value's token, and nothing else
    torch, csa, dev = _t()
    d = 64
    s = csa.make_shape(1, 1, 1, d, 128, "f32")
    cache = csa.KV4Cache(s, dev)
    rng = np.random.default_rng(9)
    k, v = rows(rng, (1, 128, 1, d), "f32"), rows(rng, (1, 128, 1, d), "f32")
    k[0, :, 0, 5] = 2.5
    v[0, 7, 0] = -1.75
    k[0, 3, 0, 9], k[0, 70, 0, 9] = float("nan"), float("inf")
    v[0, 11, 0, 2], v[0, 99, 0, 60] = float("-inf"), float("nan")
    cache.append(k, v, i64([128]))
    K, V = torch.empty(1, 1, 128, d, device=dev), torch.empty(1, 1, 128, d, device=dev)
    cache.unpack(K, V, i64([128]))
    assert bool((K[..., 5] == 2.5).all()) and bool((V[0, 0, 7] == -1.75).all())
    bad = torch.isnan(K[0, 0])
    assert bool(bad[:, 9].all()) and int(bad.sum()) == 128
    bad = torch.isnan(V[0, 0])
    assert bool(bad[11].all()) and bool(bad[99].all()) and int(bad.sum()) == 2 * d


def test_append_and_unpack_ranges_are_reported():
    torch, csa, dev = _t()
    s = csa.make_shape(3, 1, 1, 64, 100, "bf16")
    x = torch.ones(3, 70, 1, 64, dtype=torch.bfloat16, device=dev)
    for lens, new in (([101, 70, 70], [70, 70, 70]), ([70, 69, 100], [70, 70, 70]),
                      ([70, 71, 100], [70, 71, 70]), ([70, 70, 100], [70, 70, -1])):
        cache = csa.KV4Cache(s, dev)
        cache.append(x, x, i64(lens), i64(new))
        assert csa.csa_check(cache.status) == 1
        for b in range(3):
            ok = 0 <= new[b] <= 70 and new[b] <= lens[b] <= 100
            wrote = bool((cache.bounds[b] != 0).any()) or bool((cache.Kt[b] != 0).any())
            assert wrote == ok
    K = torch.full((3, 1, 10, 64), 2.0, dtype=torch.bfloat16, device=dev)
    V = K.clone()
    cache.unpack(K, V, i64([101, 70, 70]), i64([0, -1, 0]))
    assert csa.csa_check(cache.status) == 1
    assert bool((K[:2] == 2.0).all()) and not bool((V[2] == 2.0).any())
    cache.unpack(K, V, i64([0, 70, 70]), i64([0, 1 << 40, 0]))
    assert csa.csa_check(cache.status) == 0 and bool((K[0] == 2.0).all())


# ------------------------------------------------------------ attention

def check_decode(o, lse, q, model, lens, nq, G):
    """o [B][T][Hq][d], lse [B][T][Hq] against float64; rows past nq are
    not looked at."""
    B, T, Hq, d = o.shape
    worst = 0.0
    for b in range(B):
        for g in range(Hq // G):
            k, v, mag = model.stands(b, g)
            for t in range(nq[b]):
                seen = lens[b] - nq[b] + t + 1
                for h in range(g * G, (g + 1) * G):
                    ref, ls = kv4.attention(q[b, t, h], k, v, seen)
                    if seen <= 0:
                        assert np.all(o[b, t, h] == 0)
                        assert lse is None or lse[b, t, h] == -np.inf
                        continue
                    S = (mag[:seen].astype(np.float64) @ np.abs(q[b, t, h])).max() / np.sqrt(d)
                    eps = (2.0 ** -21 + 8 * np.sqrt(d) * 2.0 ** -24) * S
                    rest = 2.0 ** -20 + 8 * np.sqrt(seen) * 2.0 ** -24
                    vmax = np.abs(v[:seen]).max()
                    err = np.abs(o[b, t, h] - ref).max() / (vmax * (2 * eps + rest))
                    worst = max(worst, err)
                    assert err <= 1, (b, t, h, err)
                    if lse is not None:
                        assert abs(lse[b, t, h] - ls) <= eps + rest + 2.0 ** -22 * abs(ls), (b, t, h)
    return worst


def filled(rng, dtype, d, H, lens, n_max, Hq, step=500):
    """A cache with random rows appended up to lens, and its model."""
    _, csa, dev = _t()
    s = csa.make_shape(len(lens), Hq, H, d, n_max, dtype)
    cache, model = csa.KV4Cache(s, dev), Model(len(lens), H, d)
    # what lies past the lengths must not matter
    cache.K4.fill_(0xFF)
    cache.V4.fill_(0xFF)
    for name in ("bounds", "vscale", "Kt", "Vt"):
        getattr(cache, name).fill_(float("nan"))
    have = [0] * len(lens)
    while have != list(lens):
        new = [min(step, n - m) for n, m in zip(lens, have)]
        have = append(cache, model, rng, dtype, have, new, max(new))
    return s, cache, model


@pytest.mark.parametrize("G,T", [(1, 1), (2, 1), (4, 1), (8, 1), (4, 2), (1, 5),
                                 (2, 3), (4, 5), (8, 3), (8, 8), (1, 16), (4, 16)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("f32", 128), ("bf16", 64)])
def test_decode(G, T, dtype, d):
    torch, csa, dev = _t()
    rng = np.random.default_rng(100 * G + T + d)
    H = 2
    lens = [0, 1, 63, 64, 65, 200, 448, 1311]
    nq = [int(rng.integers(0, T + 1)) for _ in lens] if T > 1 else [1] * len(lens)
    nq[1], nq[-1] = T, T          # more tokens than positions in sequence 1
    s, cache, model = filled(rng, dtype, d, H, lens, 1400, G * H)
    q = rows(rng, (len(lens), T, G * H, d), dtype)
    q[2] *= 0.05
    q[3] *= 3.0
    op = csa.KV4Decode(s, dev, T, with_lse=True)
    op.o.fill_(55.0)
    o = op(q, cache, i64(lens), i64(nq))
    assert csa.csa_check(op.ws) == 0
    on = f64(o)
    check_decode(on, f64(op.lse), f64(q), model, lens, nq, G)
    for b in range(len(lens)):
        assert np.all(on[b, nq[b]:] == 55.0)
    # again, and on another stream: the same bits
    side = torch.cuda.Stream(dev)
    first = o.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        op(q, cache, i64(lens), i64(nq))
    torch.cuda.synchronize()
    assert torch.equal(first, o)


@pytest.mark.parametrize("dtype,d,G,lens", [
    ("bf16", 128, 4, [20011]), ("f32", 64, 8, [9000, 64 * 200, 77]),
    ("bf16", 64, 1, [4096] * 5), ("f32", 128, 2, [5000, 1])])
def test_decode_longer(dtype, d, G, lens):
    # items cut over many CTAs, joined from the workspace
    torch, csa, dev = _t()
    rng = np.random.default_rng(len(lens) + d)
    s, cache, model = filled(rng, dtype, d, 1, lens, max(lens), G, step=4096)
    q = rows(rng, (len(lens), 1, G, d), dtype)
    op = csa.KV4Decode(s, dev, 1, with_lse=True)
    op.ws.fill_(0xFF)             # contents on entry do not matter
    o = op(q, cache, i64(lens))
    assert csa.csa_check(op.ws) == 0
    check_decode(f64(o), f64(op.lse), f64(q), model, lens, [1] * len(lens), G)


@pytest.mark.parametrize("dtype,d,G,T", [
    ("bf16", 128, 4, 2), ("bf16", 64, 8, 8), ("f32", 128, 4, 5),
    ("bf16", 128, 1, 16), ("f32", 64, 2, 1)])
def test_decode_tokens_over_cut_sequences(dtype, d, G, T):
    # several query tokens, ragged, with sequences cut over CTAs at blocks
    # that some tokens see in part
    torch, csa, dev = _t()
    rng = np.random.default_rng(7 * T + G)
    lens = [0, 1, 64, 1700, 5003, 130, 4992]
    nq = [min(T, 1 + i % T) for i in range(len(lens))]
    nq[0], nq[1], nq[3] = T, T, 0
    s, cache, model = filled(rng, dtype, d, 2, lens, 5100, 2 * G, step=4096)
    q = rows(rng, (len(lens), T, 2 * G, d), dtype)
    op = csa.KV4Decode(s, dev, T, with_lse=True)
    assert op.ws_bytes > 256
    op.ws.fill_(0xFF)
    op.o.fill_(55.0)
    o = op(q, cache, i64(lens), i64(nq))
    assert csa.csa_check(op.ws) == 0
    on = f64(o)
    check_decode(on, f64(op.lse), f64(q), model, lens, nq, G)
    for b in range(len(lens)):
        assert np.all(on[b, nq[b]:] == 55.0)
    first = o.clone()
    assert torch.equal(first, op(q, cache, i64(lens), i64(nq)))


@pytest.mark.parametrize("scale", [2.0 ** -90, 2.0 ** 98])
def test_decode_extreme_magnitudes(scale):
    # up to the documented 2^100, q scaled against k
    torch, csa, dev = _t()
    rng = np.random.default_rng(77)
    d, n = 64, 64 * 3 + 11
    s = csa.make_shape(1, 4, 1, d, n, "f32")
    k = (rng.uniform(-1, 1, (1, n, 1, d)) * scale).astype(np.float32)
    v = (rng.uniform(-1, 1, (1, n, 1, d)) * scale).astype(np.float32)
    q = (rng.normal(size=(1, 1, 4, d)) / scale).astype(np.float32)
    to = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)
    cache, model = csa.KV4Cache(s, dev), Model(1, 1, d)
    cache.append(to(k), to(v), i64([n]))
    model.add(k, v, [n])
    op = csa.KV4Decode(s, dev, 1, with_lse=True)
    o = op(to(q), cache, i64([n]))
    check_decode(f64(o), f64(op.lse), q.astype(np.float64), model, [n], [1], 4)


def test_first_call_on_another_stream():
    # buffers and outputs are ready for any stream once they are made, however
    # far behind the stream is that made them
    torch, csa, dev = _t()
    rng = np.random.default_rng(5)
    lens = [90, 128]
    s = csa.make_shape(2, 4, 2, 64, 200, "bf16")
    k, v = rows(rng, (2, 128, 2, 64), "bf16"), rows(rng, (2, 128, 2, 64), "bf16")
    q = rows(rng, (2, 1, 4, 64), "bf16")
    ln = i64(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)

    def run(stream):
        cache, op = csa.KV4Cache(s, dev), csa.KV4Decode(s, dev)
        with torch.cuda.stream(stream):
            cache.append(k, v, ln, ln)
            op(q, cache, ln)
        return cache, op
    want = run(torch.cuda.current_stream())[1].o.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    cache, op = run(side)
    torch.cuda.synchronize()
    assert torch.equal(op.o, want)


def test_decode_many_short_sequences():
    torch, csa, dev = _t()
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.integers(0, 140, 128)]
    s, cache, model = filled(rng, "bf16", 64, 2, lens, 150, 4)
    q = rows(rng, (128, 1, 4, 64), "bf16")
    op = csa.KV4Decode(s, dev)
    o = op(q, cache, i64(lens))
    check_decode(f64(o), None, f64(q), model, lens, [1] * 128, 2)


def test_decode_scales_of_the_codes():
    # keys and values from 2^-30 to 2^30, block by block and token by token:
    # the scores stay moderate (q scales against k), every weight matters
    torch, csa, dev = _t()
    rng = np.random.default_rng(12)
    d, n = 128, 64 * 9 + 5
    for kscale in (2.0 ** -20, 1.0, 2.0 ** 20):
        s = csa.make_shape(1, 4, 1, d, n, "f32")
        k = rng.normal(size=(1, n, 1, d)).astype(np.float32) * kscale
        k[0, 64:128] *= 2.0 ** -6
        k[0, 128:192] *= 4.0
        v = rng.normal(size=(1, n, 1, d)).astype(np.float32)
        v *= (2.0 ** rng.integers(-9, 10, (1, n, 1, 1))).astype(np.float32)
        v[0, 70] = 0.5                 # a constant row
        q = rng.normal(size=(1, 1, 4, d)).astype(np.float32) / kscale
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)
        cache, model = csa.KV4Cache(s, dev), Model(1, 1, d)
        cache.append(to(k), to(v), i64([n]))
        model.add(k, v, [n])
        op = csa.KV4Decode(s, dev, 1, with_lse=True)
        o = op(to(q), cache, i64([n]))
        check_decode(f64(o), f64(op.lse), q.astype(np.float64), model, [n], [1], 4)


def test_decode_peaks_late_and_early():
    # the running maximum jumps by hundreds within a block, at the first and
    # at the last block, up and (elsewhere) not at all
    torch, csa, dev = _t()
    rng = np.random.default_rng(13)
    d, n = 64, 1500
    for at in (0, 63, 64, 700, 1499):
        s = csa.make_shape(1, 8, 1, d, n, "f32")
        q = rng.normal(size=(1, 1, 8, d)).astype(np.float32)
        k = 0.1 * rng.normal(size=(1, n, 1, d)).astype(np.float32)
        k[0, at, 0] = 30 * q[0, 0, 3]
        v = rng.normal(size=(1, n, 1, d)).astype(np.float32)
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)
        cache, model = csa.KV4Cache(s, dev), Model(1, 1, d)
        cache.append(to(k), to(v), i64([n]))
        model.add(k, v, [n])
        op = csa.KV4Decode(s, dev, 1)
        o = op(to(q), cache, i64([n]))
        check_decode(f64(o), None, q.astype(np.float64), model, [n], [1], 8)


@pytest.mark.parametrize("what", ["tail", "block"])
def test_decode_unseen_values_do_not_leak(what):
    # a drafted token's NaN value reaches only the rows that see it
    torch, csa, dev = _t()
    rng = np.random.default_rng(14)
    d, T, G = 128, 4, 2
    n = 200 if what == "tail" else 192
    s = csa.make_shape(1, G, 1, d, n, "bf16")
    cache = csa.KV4Cache(s, dev)
    k, v = rows(rng, (1, n, 1, d), "bf16"), rows(rng, (1, n, 1, d), "bf16")
    v[0, n - 2, 0, 17] = float("nan")
    v[0, n - 1] = float("inf")
    cache.append(k, v, i64([n]))
    q = rows(rng, (1, T, G, d), "bf16")
    op = csa.KV4Decode(s, dev, T)
    o = op(q, cache, i64([n]))
    assert torch.isfinite(o[0, :T - 2]).all()
    if what == "tail":
        assert torch.isnan(o[0, T - 2, :, 17]).all()
        assert int(torch.isnan(o[0, T - 2]).sum()) == G
    else:
        assert torch.isnan(o[0, T - 2]).all()
    assert not torch.isfinite(o[0, T - 1]).any()
    clean = v.clone()
    clean[0, n - 2:] = 0
    cache.append(k, clean, i64([n]))
    o2 = op(q, cache, i64([n])).clone()
    cache.append(k, v, i64([n]))
    assert torch.equal(op(q, cache, i64([n]))[0, :T - 2], o2[0, :T - 2])


def test_decode_strided_queries_and_ranges():
    torch, csa, dev = _t()
    rng = np.random.default_rng(15)
    d, G, H, T = 128, 4, 2, 3
    lens = [150, 64]
    s, cache, model = filled(rng, "bf16", d, H, lens, 160, G * H)
    q = rows(rng, (2, G * H, T, d), "bf16").transpose(1, 2)
    op = csa.KV4Decode(s, dev, T)
    o = op(q, cache, i64(lens)).clone()
    assert torch.equal(o, op(q.contiguous(), cache, i64(lens)))
    check_decode(f64(o), None, f64(q), model, lens, [T, T], G)
    op(q, cache, i64([150, 161]))
    assert csa.csa_check(op.ws) == 1
    op(q, cache, i64([-1, 64]))
    assert csa.csa_check(op.ws) == 1
    op(q, cache, i64(lens), i64([3, 4]))
    assert csa.csa_check(op.ws) == 1
    op(q, cache, i64(lens), i64([0, -1]))
    assert csa.csa_check(op.ws) == 1
    op(q, cache, i64(lens), i64([0, 3]))
    assert csa.csa_check(op.ws) == 0


def test_offsets_past_32_bits():
    # arrays of more than 2^31 bytes and elements: the last sequence's rows
    torch, csa, dev = _t()
    rng = np.random.default_rng(16)
    d, H, B, n_max = 128, 20, 2, 1 << 20      # K4: 2.7e9 bytes
    s = csa.make_shape(B, H, H, d, n_max, "bf16")
    cache, model = csa.KV4Cache(s, dev), Model(B, H, d)
    lens = append(cache, model, rng, "bf16", [0, 0], [3, 200], 200)
    q = rows(rng, (B, 1, H, d), "bf16")
    o = csa.KV4Decode(s, dev)(q, cache, i64(lens))
    check_decode(f64(o), None, f64(q), model, lens, [1, 1], 1)
    K = torch.zeros(B, H, 130, d, dtype=torch.bfloat16, device=dev)
    V = torch.zeros_like(K)
    cache.unpack(K, V, i64(lens), i64([0, 60]))
    k, v, _ = model.stands(1, H - 1)
    assert torch.equal(K[1, H - 1].cpu(), torch.from_numpy(k[60:190]).bfloat16())
    assert torch.equal(V[1, H - 1].cpu(), torch.from_numpy(v[60:190]).bfloat16())
    del cache
    # the last rows of a sequence of 2^20 tokens, in their far blocks
    s = csa.make_shape(1, 2, 2, d, n_max, "bf16")
    cache = csa.KV4Cache(s, dev)
    x = rows(rng, (1, 70, 2, d), "bf16")
    cache.append(x, x, i64([n_max]), i64([70]))
    K = torch.zeros(1, 2, 70, d, dtype=torch.bfloat16, device=dev)
    cache.unpack(K, K.clone(), i64([n_max]), i64([n_max - 70]))
    c, _, m, dl = quantize_keys(float32(x)[0, 6:, 1], BLOCK)
    want = torch.from_numpy(kv4.stands_for(c, m[0], dl[0])).bfloat16()
    assert torch.equal(K[0, 1, 6:].cpu(), want)
    # the 16-bit cache behind the rotation: 2^31 elements and more
    big = csa.make_shape(2, 8, 8, d, n_max + 7, "bf16")
    Kc = torch.zeros(2, 8, n_max + 7, d, dtype=torch.bfloat16, device=dev)
    Vc = torch.zeros_like(Kc)
    x = rows(rng, (2, 2, 8, d), "bf16")
    csa.QKNormRope(big, dev)(x, x, x, Kc, Vc, i64([2, n_max + 7]))
    assert torch.equal(Kc[1, 7, -2:], x[1, :, 7]) and torch.equal(Vc[1, 7, -2:], x[1, :, 7])
    assert int(Kc.count_nonzero(dim=3).count_nonzero()) == 2 * 2 * 8


# ------------------------------------------------- the operators together

def test_layers_decoded_with_one_graph():
    # Two layers: a prompt of uneven lengths, then tokens one by one with one
    # captured graph (norms and rotation, append, attention), lengths on the
    # device; every token against float64 on the rows the cache stands for.
    torch, csa, dev = _t()
    rng = np.random.default_rng(21)
    B, Hq, H, d, n_max, P, steps = 3, 8, 2, 128, 300, 130, 9
    G = Hq // H
    s = csa.make_shape(B, Hq, H, d, n_max, "bf16")
    f = 500000.0 ** (-np.arange(d // 2) / (d // 2))
    start = [130, 60, 124]                       # blocks fill on the way
    layers = []
    for _ in range(2):
        w = rows(rng, (d,), "bf16")
        layers.append(dict(
            rope=csa.QKNormRope(s, dev, w, w, inv_freq=f),
            cache=csa.KV4Cache(s, dev), model=Model(B, H, d),
            dec=csa.KV4Decode(s, dev),
            x=torch.zeros(B, 1, Hq + 2 * H, d, dtype=torch.bfloat16, device=dev),
            q=torch.zeros(B, 1, Hq, d, dtype=torch.bfloat16, device=dev),
            k=torch.zeros(B, 1, H, d, dtype=torch.bfloat16, device=dev),
            v=torch.zeros(B, 1, H, d, dtype=torch.bfloat16, device=dev)))
    lens = i64(start)
    for ly in layers:
        x = rows(rng, (B, P, Hq + 2 * H, d), "bf16")
        k = torch.zeros(B, P, H, d, dtype=torch.bfloat16, device=dev)
        v = torch.zeros_like(k)
        ly["rope"](x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:], k, v,
                   lens, lens, to_cache=False)
        ly["cache"].append(k, v, lens, lens)
        ly["model"].add(float32(k), float32(v), start)

    def token():
        for ly in layers:
            x = ly["x"]
            ly["rope"](x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:],
                       ly["k"], ly["v"], lens, to_cache=False, q_out=ly["q"])
            ly["cache"].append(ly["k"], ly["v"], lens)
            ly["dec"](ly["q"], ly["cache"], lens)

    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    graph = None
    for t in range(steps):
        lens += 1
        for ly in layers:
            ly["x"].copy_(rows(rng, tuple(ly["x"].shape), "bf16"))
        torch.cuda.synchronize()
        if t == 0:
            with torch.cuda.stream(side):
                token()                          # eager
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    token()
            graph.replay()
        torch.cuda.synchronize()
        now = [a + t + 1 for a in start]
        for ly in layers:
            ly["model"].add(float32(ly["k"]), float32(ly["v"]), [1] * B)
            assert csa.csa_check(ly["dec"].ws) == 0
            assert csa.csa_check(ly["cache"].status) == 0
            xn, qn = f64(ly["x"]), f64(ly["q"])
            w = f64(ly["rope"].weights[0])
            for b in range(B):
                for h in range(Hq):
                    check_rope(qn[b, 0, h], xn[b, 0, h], w, now[b] - 1, f, False, 1e-6, "bf16")
            check_decode(f64(ly["dec"].o), None, qn, ly["model"], now, [1] * B, G)


def test_rope_feeds_the_certified_step():
    # the rotated rows land where csa_quantize_keys and the decode step read
    # them: the step's fallback-free output equals dense attention within its
    # bound, and dense attention the definition
    torch, csa, dev = _t()
    rng = np.random.default_rng(22)
    B, Hq, H, d, n = 1, 4, 1, 128, 500
    s = csa.make_shape(B, Hq, H, d, n, "bf16")
    f = 10000.0 ** (-np.arange(d // 2) / (d // 2))
    rope = csa.QKNormRope(s, dev, inv_freq=f)
    x = rows(rng, (B, n, Hq + 2 * H, d), "bf16") * 0.5
    K = torch.zeros(B, H, n, d, dtype=torch.bfloat16, device=dev)
    V = torch.zeros_like(K)
    q = rope(x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:], K, V, i64([n]))
    last = q[:, -1].contiguous()
    meta = csa.meta_buffers(s, dev)
    csa.check(csa.csa_quantize_keys(s, K, V, [n], 0, *meta))
    step = csa.DecodeStep(s, csa.make_params(), dev)
    o, beta, _, _ = step(last, K, V, meta, [n], [7])
    dense = csa.DenseDecode(s, dev)(last, K, V, [n])
    torch.cuda.synchronize()
    err = (o - dense).norm(dim=-1)
    assert bool((err <= beta * (1 + 2e-3) + 2e-3 * dense.norm(dim=-1)).all())
    ref, _ = kv4.attention(f64(last)[0, 2], f64(K)[0, 0], f64(V)[0, 0], n)
    assert np.abs(f64(dense)[0, 2] - ref).max() <= 1e-5 * np.abs(f64(V)).max()


@pytest.mark.parametrize("rot,inter", [(24, False), (104, False), (40, True), (16, False), (128, False)])
def test_rope_bf16_odd_rotations_and_many_heads(rot, inter):
    # rotated parts that do not divide into 16-byte vectors; enough tokens for
    # several heads to a group of lanes
    torch, csa, dev = _t()
    rng = np.random.default_rng(rot)
    B, T, Hq, Hkv, d = 2, 700, 20, 5, 128
    s = csa.make_shape(B, Hq, Hkv, d, 800, "bf16")
    f = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    wq, wk = rows(rng, (d,), "bf16"), rows(rng, (d,), "bf16")
    op = csa.QKNormRope(s, dev, wq, wk, inv_freq=f, interleaved=inter)
    q, k, v = [rows(rng, (B, T, h, d), "bf16") for h in (Hq, Hkv, Hkv)]
    K = torch.zeros(B, Hkv, 800, d, dtype=torch.bfloat16, device=dev)
    V = torch.zeros_like(K)
    qo = op(q, k, v, K, V, i64([800, 705]))
    qn, kn, qx, kx = f64(qo), f64(K), f64(q), f64(k)
    for b, t in ((0, 0), (0, 699), (1, 350), (1, 699)):
        pos = (100 if b == 0 else 5) + t
        for h in range(Hq):
            check_rope(qn[b, t, h], qx[b, t, h], f64(wq), pos, f, inter, 1e-6, "bf16")
        for g in range(Hkv):
            check_rope(kn[b, g, pos], kx[b, t, g], f64(wk), pos, f, inter, 1e-6, "bf16")
    assert torch.equal(V[0, :, 100:], v[0].transpose(0, 1))
    assert torch.equal(V[1, :, 5:705], v[1].transpose(0, 1))
