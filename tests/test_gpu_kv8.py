"""The 8-bit K/V cache on the GPU (csa_kv8_append, csa_kv8_unpack, csa_kv8_decode),
against the plain restatement in oracle/kv8.py and float64 attention.

Tolerances are derived, not fitted:
  * codes, steps and spans: bit for bit; rows read back: the float32 value,
    rounded once to the type, bit for bit;
  * attention: a score's rounding error is at most eps_s = (2^-21 + 8 sqrt(d)
    2^-24) S, S = max over tokens of sum_c |q_c k_c| / sqrt(d) (products to 22
    bits, and d roundings of independent sign at eight standard deviations); it
    moves every weight by a factor within exp(+-eps_s), so the output by at most
    2 eps_s vmax; the weights and sums over n tokens add (2^-20 + 8 sqrt(n)
    2^-24) vmax, vmax the largest |v| stood for.
"""
import numpy as np
import pytest

from oracle import kv4, kv8
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


def float32(t):
    return t.detach().float().cpu().numpy()


def rows(rng, size, dtype):
    """Random rows with a few strong channels, in the type."""
    torch, _, dev = _t()
    x = rng.normal(size=size).astype(np.float32)
    x[..., :3] *= 6
    return torch.from_numpy(x).to(dev).to(tdtype(dtype))


def on_gpu(x):
    torch, _, dev = _t()
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)


class Model:
    """The rows appended so far, per sequence and KV head."""

    def __init__(self, B, H, d):
        self.k = [[np.zeros((0, d), np.float32) for _ in range(H)] for _ in range(B)]
        self.v = [[np.zeros((0, d), np.float32) for _ in range(H)] for _ in range(B)]

    def add(self, k, v, new):
        for b, m in enumerate(new):
            for g in range(len(self.k[b])):
                self.k[b][g] = np.concatenate([self.k[b][g], k[b, :m, g]])
                self.v[b][g] = np.concatenate([self.v[b][g], v[b, :m, g]])

    def blocks(self, b, g):
        """(K8, V8, scale, span) of every whole block."""
        k, v = self.k[b][g], self.v[b][g]
        return [kv8.block(k[j:j + BLOCK], v[j:j + BLOCK]) for j in range(0, len(k) - BLOCK + 1, BLOCK)]

    def stands(self, b, g):
        """float32 rows K, V."""
        k, v = self.k[b][g].copy(), self.v[b][g].copy()
        for x in (k, v):
            for j in range(0, len(x) - BLOCK + 1, BLOCK):
                step = kv8.steps(x[j:j + BLOCK])
                x[j:j + BLOCK] = kv8.stands_for(kv8.codes(x[j:j + BLOCK], step), step)
        return k, v


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


def spoil(cache):
    """What lies past the lengths must not matter."""
    for name in ("K8", "V8", "span"):
        getattr(cache, name).fill_(0xFF)
    for name in ("scale", "Kt", "Vt"):
        getattr(cache, name).fill_(float("nan"))


def filled(rng, dtype, d, H, lens, n_max, Hq, step=500):
    """A cache with random rows appended up to lens, and its model."""
    _, csa, dev = _t()
    s = csa.make_shape(len(lens), Hq, H, d, n_max, dtype)
    cache, model = csa.KV8Cache(s, dev), Model(len(lens), H, d)
    spoil(cache)
    have = [0] * len(lens)
    while have != list(lens):
        new = [min(step, n - m) for n, m in zip(lens, have)]
        have = append(cache, model, rng, dtype, have, new, max(new))
    return s, cache, model


# ------------------------------------------------------- append and unpack

@pytest.mark.parametrize("dtype,d,H", [("bf16", 128, 2), ("f32", 64, 3),
                                       ("bf16", 64, 1), ("f32", 128, 1)])
def test_append_and_unpack_bit_for_bit(dtype, d, H):
    torch, csa, dev = _t()
    rng = np.random.default_rng(d + H)
    B, n_max = 3, 400
    s = csa.make_shape(B, H, H, d, n_max, dtype)
    cache = csa.KV8Cache(s, dev)
    for name in ("K8", "V8", "span"):
        getattr(cache, name).fill_(0xA5)
    for name in ("scale", "Kt", "Vt"):
        getattr(cache, name).fill_(-77.0)
    model, lens = Model(B, H, d), [0] * B
    for new in ([1, 0, 64], [62, 63, 1], [1, 2, 0], [0, 0, 0], [65, 1, 127],
                [130, 61, 64], [7, 1, 130]):
        lens = append(cache, model, rng, dtype, lens, new, max(1, max(new)))
        assert csa.csa_check(cache.status) == 0
        nblk = cache.scale.shape[2]
        have = [x.cpu().numpy().reshape((B, H, nblk) + size) for x, size in (
            (cache.K8, (BLOCK * d,)), (cache.V8, (d, BLOCK)), (cache.scale, (2,)), (cache.span, (2, d)))]
        Kt, Vt = float32(cache.Kt), float32(cache.Vt)
        for b in range(B):
            w = lens[b] // BLOCK
            for g in range(H):
                for j, want in enumerate(model.blocks(b, g)):
                    for x, y in zip(have, want):
                        assert np.array_equal(x[b, g, j], y)
                # nothing past the whole blocks is written
                for x, y in zip(have, (0xA5, 0xA5, -77, 0xA5)):
                    assert np.all(x[b, g, w:] == y)
                r = lens[b] % BLOCK
                assert np.array_equal(Kt[b, g, :r], model.k[b][g][w * BLOCK:])
                assert np.array_equal(Vt[b, g, :r], model.v[b][g][w * BLOCK:])
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
                    for got, want, rest in zip((K, V), model.stands(b, g), (3.0, 4.0)):
                        want = torch.from_numpy(want[f:f + m]).to(tdtype(dtype))
                        assert torch.equal(got[b, g, :m].cpu(), want)
                        assert bool((got[b, g, m:] == rest).all())


def test_append_takes_any_strides():
    # operands cut from one projection, heads-major ones, and a broadcast one
    torch, csa, dev = _t()
    rng = np.random.default_rng(4)
    B, T, H, d = 2, 150, 3, 64
    s = csa.make_shape(B, H, H, d, 200, "bf16")
    both = rows(rng, (B, T, 2 * H, d), "bf16")
    k, v = both[:, :, :H], both[:, :, H:]
    made = []
    for a, b in ((k, v), (k.contiguous(), v.contiguous()),
                 (k.transpose(1, 2).contiguous().transpose(1, 2), v.transpose(1, 2).contiguous().transpose(1, 2))):
        cache = csa.KV8Cache(s, dev)
        cache.append(a, b, i64([150, 131]), i64([150, 131]))
        made.append(cache)
    one = csa.KV8Cache(s, dev)
    one.append(k[:, :, :1].expand(B, T, H, d), v[:1].expand(B, T, H, d), i64([150, 150]))
    for x in ("K8", "V8", "scale", "span", "Kt", "Vt"):
        assert torch.equal(getattr(made[0], x), getattr(made[1], x))
        assert torch.equal(getattr(made[0], x), getattr(made[2], x))
    assert torch.equal(one.K8[:, 0], one.K8[:, 2]) and torch.equal(one.V8[0], one.V8[1])
    assert torch.equal(one.K8[0, 0, :2], made[0].K8[0, 0, :2])


def test_append_special_values():
    # a NaN or infinity spoils the keys or the values of its block, and nothing
    # else; blocks of zeros, of subnormal numbers, of the largest ones
    torch, csa, dev = _t()
    d = 64
    s = csa.make_shape(1, 1, 1, d, 64 * 6, "f32")
    cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
    rng = np.random.default_rng(9)
    k, v = [rng.normal(size=(1, 64 * 6, 1, d)).astype(np.float32) for _ in range(2)]
    k[0, 3, 0, 9], k[0, 70, 0, 9] = np.nan, np.inf
    v[0, 130, 0, 2], v[0, 99, 0, 60] = -np.inf, np.nan
    k[0, 192:256], v[0, 192:256] = 0.0, -0.0
    k[0, 256:320] *= np.float32(2.0 ** -146)
    v[0, 256:320] *= np.float32(2.0 ** -129)
    k[0, 320:] = np.clip(k[0, 320:] * np.float32(2.0 ** 127), -3e38, 3e38)
    v[0, 320:, 0, :] = 1.0
    cache.append(on_gpu(k), on_gpu(v), i64([64 * 6]))
    model.add(k, v, [64 * 6])
    K, V = [torch.empty(1, 1, 64 * 6, d, device=dev) for _ in range(2)]
    cache.unpack(K, V, i64([64 * 6]))
    K, V = float32(K)[0, 0], float32(V)[0, 0]
    assert np.all(np.isnan(K[:128])) and not np.any(np.isnan(K[128:]))
    assert np.all(np.isnan(V[64:192])) and not np.any(np.isnan(V[:64])) and not np.any(np.isnan(V[192:]))
    want = model.stands(0, 0)
    assert np.array_equal(K[128:], want[0][128:]) and np.array_equal(V[192:], want[1][192:])
    assert np.all(K[192:256] == 0) and np.all(V[320:] == 1.0)
    for j, (_, _, scale, span) in enumerate(model.blocks(0, 0)):
        assert np.array_equal(cache.scale[0, 0, j].cpu().numpy(), scale, equal_nan=True)
        assert np.array_equal(cache.span[0, 0, j].cpu().numpy(), span)


def test_append_halves_are_rounded_to_even():
    # steps of a power of two and values half way between two codes
    torch, csa, dev = _t()
    d = 128
    for dtype in ("bf16", "f32"):
        s = csa.make_shape(1, 1, 1, d, 64, dtype)
        x = np.random.default_rng(1).integers(-253, 254, (1, 64, 1, d)).astype(np.float32) / 2
        x[0, 5, 0, 7] = -127.0
        x = np.clip(x, -126.5, 126.5)
        x[0, 5, 0, 7] = -127.0
        t = on_gpu(x * 2.0 ** -5).to(tdtype(dtype))
        cache = csa.KV8Cache(s, dev)
        cache.append(t, t, i64([64]))
        k8, v8, scale, span = kv8.block(float32(t)[0, :, 0], float32(t)[0, :, 0])
        assert np.array_equal(cache.K8.cpu().numpy().ravel(), k8) and np.array_equal(cache.V8.cpu().numpy()[0, 0, 0], v8)
        assert scale[0] == 2.0 ** -5 and np.array_equal(cache.span.cpu().numpy()[0, 0, 0], span)


def test_append_and_unpack_ranges_are_reported():
    torch, csa, dev = _t()
    s = csa.make_shape(3, 1, 1, 64, 100, "bf16")
    x = torch.ones(3, 70, 1, 64, dtype=torch.bfloat16, device=dev)
    for lens, new in (([101, 70, 70], [70, 70, 70]), ([70, 69, 100], [70, 70, 70]),
                      ([70, 71, 100], [70, 71, 70]), ([70, 70, 100], [70, 70, -1])):
        cache = csa.KV8Cache(s, dev)
        cache.append(x, x, i64(lens), i64(new))
        assert csa.csa_check(cache.status) == 1 and csa.csa_check(cache.refused) == 1
        for b in range(3):
            ok = 0 <= new[b] <= 70 and new[b] <= lens[b] <= 100
            wrote = bool((cache.scale[b] != 0).any()) or bool((cache.Kt[b] != 0).any())
            assert wrote == ok
        cache.append(x, x, i64([70, 70, 70]))
        assert csa.csa_check(cache.status) == 0 and csa.csa_check(cache.refused) == 1
        cache.refused.zero_()
        cache.append(x, x, i64([70, 70, 70]))
        assert csa.csa_check(cache.refused) == 0
    K = torch.full((3, 1, 10, 64), 2.0, dtype=torch.bfloat16, device=dev)
    V = K.clone()
    cache.unpack(K, V, i64([101, 70, 70]), i64([0, -1, 0]))
    assert csa.csa_check(cache.status) == 1
    assert bool((K[:2] == 2.0).all()) and not bool((V[2] == 2.0).any())
    cache.unpack(K, V, i64([0, 70, 70]), i64([0, 1 << 40, 0]))
    assert csa.csa_check(cache.status) == 0 and bool((K[0] == 2.0).all())


# ------------------------------------------------------------ attention

def check_row(o, lse, q, k, v, what):
    """One row against float64 attention over the rows k, v; the error as a
    share of the tolerance."""
    d = len(q)
    ref, ls = kv4.attention(q, k, v, len(k))
    if len(k) == 0:
        assert np.all(o == 0) and (lse is None or lse == -np.inf), what
        return 0.0
    S = (np.abs(k).astype(np.float64) @ np.abs(q)).max() / np.sqrt(d)
    eps = (2.0 ** -21 + 8 * np.sqrt(d) * 2.0 ** -24) * S
    rest = 2.0 ** -20 + 8 * np.sqrt(len(k)) * 2.0 ** -24
    err = np.abs(o - ref).max() / (np.abs(v).max() * (2 * eps + rest))
    assert err <= 1, (what, err)
    if lse is not None:
        assert abs(lse - ls) <= eps + rest + 2.0 ** -22 * abs(ls), what
    return err


def check_decode(o, lse, q, model, lens, nq, G):
    """o [B][T][Hq][d], lse [B][T][Hq] against float64; rows past nq are
    not looked at."""
    B, T, Hq, d = o.shape
    for b in range(B):
        for g in range(Hq // G):
            k, v = model.stands(b, g)
            for t in range(nq[b]):
                seen = max(0, lens[b] - nq[b] + t + 1)
                for h in range(g * G, (g + 1) * G):
                    check_row(o[b, t, h], None if lse is None else lse[b, t, h], q[b, t, h], k[:seen], v[:seen], (b, t, h))


@pytest.mark.parametrize("G,T", [(1, 1), (2, 1), (4, 1), (8, 1), (4, 2), (1, 5),
                                 (2, 3), (4, 5), (8, 3), (8, 8), (1, 16), (4, 16),
                                 (8, 2), (8, 4), (8, 6), (8, 7)])
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
    op = csa.KV8Decode(s, dev, T, with_lse=True)
    op.o.fill_(55.0)
    op.ws.fill_(0xFF)             # contents on entry do not matter
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
@pytest.mark.parametrize("n_max", [0, 70000])
def test_decode_longer(dtype, d, G, lens, n_max):
    # items cut over many CTAs, joined from the workspace (always with room for 70000
    # tokens), or shared by a few
    torch, csa, dev = _t()
    rng = np.random.default_rng(len(lens) + d)
    s, cache, model = filled(rng, dtype, d, 1, lens, max(lens + [n_max]), G, step=4096)
    q = rows(rng, (len(lens), 1, G, d), dtype)
    op = csa.KV8Decode(s, dev, 1, with_lse=True)
    assert op.ws_bytes > 256 or not n_max
    op.ws.fill_(0xFF)
    o = op(q, cache, i64(lens))
    assert csa.csa_check(op.ws) == 0
    check_decode(f64(o), f64(op.lse), f64(q), model, lens, [1] * len(lens), G)


@pytest.mark.parametrize("dtype,d,G,T", [
    ("bf16", 128, 4, 2), ("bf16", 64, 8, 8), ("f32", 128, 4, 5),
    ("bf16", 128, 1, 16), ("f32", 64, 2, 1), ("bf16", 128, 8, 3)])
@pytest.mark.parametrize("n_max", [5100, 30000])
def test_decode_tokens_over_cut_sequences(dtype, d, G, T, n_max):
    # several query tokens, ragged, with sequences cut over CTAs at blocks
    # that some tokens see in part (always with room for 30000 tokens), or shared
    torch, csa, dev = _t()
    rng = np.random.default_rng(7 * T + G)
    lens = [0, 1, 64, 1700, 5003, 130, 4992]
    nq = [min(T, 1 + i % T) for i in range(len(lens))]
    nq[0], nq[1], nq[3] = T, T, 0
    s, cache, model = filled(rng, dtype, d, 2, lens, n_max, 2 * G, step=4096)
    q = rows(rng, (len(lens), T, 2 * G, d), dtype)
    op = csa.KV8Decode(s, dev, T, with_lse=True)
    assert op.ws_bytes > 256 or n_max == 5100
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


@pytest.mark.parametrize("dtype,d,H,G,T,lens", [
    ("bf16", 128, 1, 4, 1, [1400]), ("f32", 64, 1, 2, 5, [64 * 31 + 63]), ("bf16", 64, 2, 8, 2, [700, 1300]),
    ("f32", 128, 3, 4, 4, [0, 1, 65, 1000, 1407]), ("bf16", 128, 8, 8, 8, [520, 64]), ("bf16", 128, 7, 1, 3, [1291] * 10),
    ("f32", 64, 2, 8, 7, [830] * 3), ("bf16", 128, 4, 8, 1, [1408, 5, 1344, 1345])])
def test_decode_items_shared_by_ctas(dtype, d, H, G, T, lens):
    # two, four or eight CTAs to an item: the fewest blocks there can be to each, shares
    # without any, idle sequences, the incomplete block beside them
    torch, csa, dev = _t()
    rng = np.random.default_rng(100 * T + len(lens))
    n_max = max(lens) + 7
    nq = [i * 5 % (T + 1) for i in range(len(lens))]
    nq[0] = T
    s, cache, model = filled(rng, dtype, d, H, lens, n_max, H * G, step=1024)
    q = rows(rng, (len(lens), T, H * G, d), dtype)
    op = csa.KV8Decode(s, dev, T, with_lse=True)
    assert op.ws_bytes == 256
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
    cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
    cache.append(on_gpu(k), on_gpu(v), i64([n]))
    model.add(k, v, [n])
    op = csa.KV8Decode(s, dev, 1, with_lse=True)
    o = op(on_gpu(q), cache, i64([n]))
    check_decode(f64(o), f64(op.lse), q.astype(np.float64), model, [n], [1], 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_blocks_of_uneven_steps(dtype):
    # keys and values from 2^-20 to 2^20 by block: the scores stay moderate
    # where q is scaled against k, and every block's weight matters; then large
    # values behind no weight, and small ones behind all of it
    torch, csa, dev = _t()
    rng = np.random.default_rng(12)
    d, n = 128, 64 * 9 + 5
    for kscale in (2.0 ** -20, 1.0, 2.0 ** 20):
        s = csa.make_shape(1, 4, 1, d, n, dtype)
        k = rng.normal(size=(1, n, 1, d)).astype(np.float32) * kscale
        k[0, 64:128] *= 2.0 ** -6
        k[0, 128:192] *= 4.0
        v = rng.normal(size=(1, n, 1, d)).astype(np.float32)
        v *= np.repeat(2.0 ** rng.integers(-20, 1, 10), 64)[:n, None, None].astype(np.float32)
        q = rng.normal(size=(1, 1, 4, d)).astype(np.float32) / kscale
        k, v, q = [on_gpu(x).to(tdtype(dtype)) for x in (k, v, q)]
        cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
        cache.append(k, v, i64([n]))
        model.add(float32(k), float32(v), [n])
        op = csa.KV8Decode(s, dev, 1, with_lse=True)
        o = op(q, cache, i64([n]))
        check_decode(f64(o), f64(op.lse), f64(q), model, [n], [1], 4)


def test_decode_small_values_under_the_weight():
    # the block that has the weight holds values 2^-20 of the others': the
    # output is held relative to them, not to the largest value there is
    torch, csa, dev = _t()
    rng = np.random.default_rng(18)
    d, n = 128, 64 * 6
    s = csa.make_shape(1, 2, 1, d, n, "f32")
    q = rng.normal(size=(1, 1, 2, d)).astype(np.float32)
    q[0, 0, 1] = q[0, 0, 0]
    k = 0.01 * rng.normal(size=(1, n, 1, d)).astype(np.float32)
    k[0, 128:192, 0] += 0.8 * q[0, 0, 0]
    v = rng.normal(size=(1, n, 1, d)).astype(np.float32)
    v[0, 128:192] *= 2.0 ** -20
    cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
    cache.append(on_gpu(k), on_gpu(v), i64([n]))
    model.add(k, v, [n])
    o = f64(csa.KV8Decode(s, dev)(on_gpu(q), cache, i64([n])))[0, 0]
    K, V = [x.astype(np.float64) for x in model.stands(0, 0)]
    for h in range(2):
        x = K @ q[0, 0, h].astype(np.float64) / np.sqrt(d)
        w = np.exp(x - x.max())
        w /= w.sum()
        S = (np.abs(K) @ np.abs(q[0, 0, h]).astype(np.float64)).max() / np.sqrt(d)
        eps = (2.0 ** -21 + 8 * np.sqrt(d) * 2.0 ** -24) * S
        # every token's own share of the error
        lim = (2 * eps + 2.0 ** -20 + 8 * np.sqrt(n) * 2.0 ** -24) * (w @ np.abs(V))
        assert w[128:192].sum() > 0.99 and np.all(np.abs(o[h] - w @ V) <= lim)


def test_decode_small_query_channels():
    # channels in which the query is 2^-20 of its largest count in full where
    # the keys are zero in the large one
    torch, csa, dev = _t()
    rng = np.random.default_rng(19)
    d, n = 64, 64 * 3
    for dtype in ("f32", "bf16"):
        s = csa.make_shape(1, 1, 1, d, n, dtype)
        k, v = [rng.normal(size=(1, n, 1, d)).astype(np.float32) for _ in range(2)]
        k[..., 5] = 0.0
        q = rng.normal(size=(1, 1, 1, d)).astype(np.float32)
        q[..., 5] = 2.0 ** 20
        k, v, q = [on_gpu(x).to(tdtype(dtype)) for x in (k, v, q)]
        cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
        cache.append(k, v, i64([n]))
        model.add(float32(k), float32(v), [n])
        op = csa.KV8Decode(s, dev, 1, with_lse=True)
        o = op(q, cache, i64([n]))
        check_decode(f64(o), f64(op.lse), f64(q), model, [n], [1], 1)


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
        cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
        cache.append(on_gpu(k), on_gpu(v), i64([n]))
        model.add(k, v, [n])
        o = csa.KV8Decode(s, dev, 1)(on_gpu(q), cache, i64([n]))
        check_decode(f64(o), None, q.astype(np.float64), model, [n], [1], 8)


def test_decode_many_short_sequences():
    torch, csa, dev = _t()
    rng = np.random.default_rng(31)
    lens = [int(x) for x in rng.integers(0, 140, 128)]
    s, cache, model = filled(rng, "bf16", 64, 2, lens, 150, 4)
    q = rows(rng, (128, 1, 4, 64), "bf16")
    o = csa.KV8Decode(s, dev)(q, cache, i64(lens))
    check_decode(f64(o), None, f64(q), model, lens, [1] * 128, 2)


@pytest.mark.parametrize("what", ["tail", "block"])
def test_decode_unseen_values_do_not_leak(what):
    # a drafted token's NaN value reaches only the rows that see it, or that see
    # part of its whole block
    torch, csa, dev = _t()
    rng = np.random.default_rng(14)
    d, T, G = 128, 4, 2
    n = 200 if what == "tail" else 192
    s = csa.make_shape(1, G, 1, d, n, "bf16")
    cache = csa.KV8Cache(s, dev)
    k, v = rows(rng, (1, n, 1, d), "bf16"), rows(rng, (1, n, 1, d), "bf16")
    v[0, n - 2, 0, 17] = float("nan")
    v[0, n - 1] = float("inf")
    cache.append(k, v, i64([n]))
    q = rows(rng, (1, T, G, d), "bf16")
    op = csa.KV8Decode(s, dev, T)
    o = op(q, cache, i64([n]))
    if what == "tail":
        assert torch.isfinite(o[0, :T - 2]).all()
        assert torch.isnan(o[0, T - 2, :, 17]).all()
        assert int(torch.isnan(o[0, T - 2]).sum()) == G
    assert not torch.isfinite(o[0, T - 1]).any()


def keys_of_the_last_block(dtype, d, G, T, n, n_max, put, seed):
    """Attention over n tokens of which put(q, k, v) changes rows first; o, lse, q and
    the rows the cache stands for."""
    torch, csa, dev = _t()
    rng = np.random.default_rng(seed)
    s = csa.make_shape(1, G, 1, d, n_max, dtype)
    k, v, q = [float32(rows(rng, (1, x, h, d), dtype)) for x, h in ((n, 1), (n, 1), (T, G))]
    put(q[0], k[0, :, 0], v[0, :, 0])
    cache, model = csa.KV8Cache(s, dev), Model(1, 1, d)
    k, v, q = [on_gpu(x).to(tdtype(dtype)) for x in (k, v, q)]
    cache.append(k, v, i64([n]))
    model.add(float32(k), float32(v), [n])
    op = csa.KV8Decode(s, dev, T, with_lse=True)
    o = op(q, cache, i64([n]))
    assert csa.csa_check(op.ws) == 0
    return f64(o)[0], f64(op.lse)[0], f64(q)[0], model.stands(0, 0)


@pytest.mark.parametrize("G,T,n,n_max", [(4, 1, 127, 128), (1, 1, 65, 9000), (4, 1, 1, 64), (8, 2, 200, 200), (4, 5, 1003, 9000),
                                         (8, 3, 700, 700), (8, 8, 72, 9000)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("f32", 128), ("bf16", 64)])
def test_infinite_keys_of_the_incomplete_block(G, T, n, n_max, dtype, d):
    # a score of -infinity is a weight of 0 (nothing is attended to where there is no
    # other), one of +infinity or a NaN makes the row NaN, and a row that does not see
    # the token is as it would be
    first = n // 64 * 64
    at = sorted({first, (first + n) // 2, n - 2, n - 1} & set(range(first, n)))

    def put(q, k, v):
        for i, p in enumerate(at):
            k[p, 7 + i % 2] = (np.inf, -np.inf)[i % 2]
        # most rows score the tokens -infinity, a few +infinity, one both in one token
        q[..., 7], q[..., 8] = -np.abs(q[..., 7]) - 0.1, np.abs(q[..., 8]) + 0.1
        q[-1, G // 2, 7] = 0.25
        if T > 1:
            q[0, 0, 8] = -0.5
            q[1, 0, 7] = 0.0

    o, lse, q, (k, v) = keys_of_the_last_block(dtype, d, G, T, n, n_max, put, d + T)
    for t in range(T):
        seen = n - T + t + 1
        for h in range(G):
            with np.errstate(invalid="ignore"):
                score = k[:seen].astype(np.float64) @ q[t, h]
            if np.isnan(score).any() or (score == np.inf).any():
                assert np.isnan(o[t, h]).all() and np.isnan(lse[t, h])
            else:
                there = score > -np.inf
                check_row(o[t, h], lse[t, h], q[t, h], k[:seen][there], v[:seen][there], (t, h))


@pytest.mark.parametrize("G,T,d", [(2, 4, 64), (8, 3, 128), (8, 8, 64), (4, 4, 128)])
@pytest.mark.parametrize("n,n_max", [(200, 200), (1001, 9000)])
def test_largest_numbers_of_the_incomplete_block(G, T, d, n, n_max):
    # float32 values that bf16 rounds to infinity, and a key of that size where the
    # query is 0: rows that do not see them are as they would be, and so is the weight
    # of the others
    top = np.finfo(np.float32).max

    def put(q, k, v):
        k[n - 3, 11], q[..., 11] = top, 0.0
        k[n - 2:] = 0.0
        v[n - 2, 9], v[n - 1, 5], v[n - 1, d - 1] = np.float32(2.0 ** 127 * (2 - 2.0 ** -8)), -top, top

    o, lse, q, (k, v) = keys_of_the_last_block("f32", d, G, T, n, n_max, put, d + T)
    for t in range(T):
        seen = n - T + t + 1
        for h in range(G):
            assert np.isfinite(o[t, h]).all()
            check_row(o[t, h], lse[t, h], q[t, h], k[:seen], v[:seen], (t, h))


def test_drafts_over_the_end_of_a_block_do_not_leak():
    # eight drafted tokens fill a block's end, eight more begin the next: those
    # of NaN keys and infinite values do not reach the ones before
    torch, csa, dev = _t()
    d, T, G, n = 64, 16, 2, 1224
    s = csa.make_shape(1, G, 1, d, n, "bf16")
    q = rows(np.random.default_rng(15), (1, T, G, d), "bf16")
    op, out = csa.KV8Decode(s, dev, T), []
    k, v = [rows(np.random.default_rng(x), (1, n, 1, d), "bf16") for x in (1, 2)]
    for bad in (False, True):
        if bad:
            k[0, n - 8:], v[0, n - 8:] = float("nan"), float("inf")
        cache = csa.KV8Cache(s, dev)
        cache.append(k, v, i64([n]))
        out.append(op(q, cache, i64([n])).clone())
    assert torch.isfinite(out[0]).all()
    assert torch.equal(out[0][0, :8], out[1][0, :8])
    assert not torch.isfinite(out[1][0, 8:]).any()


def test_decode_strided_queries_and_ranges():
    torch, csa, dev = _t()
    rng = np.random.default_rng(15)
    d, G, H, T = 128, 4, 2, 3
    lens = [150, 64]
    s, cache, model = filled(rng, "bf16", d, H, lens, 160, G * H)
    q = rows(rng, (2, G * H, T, d), "bf16").transpose(1, 2)
    op = csa.KV8Decode(s, dev, T)
    o = op(q, cache, i64(lens)).clone()
    assert torch.equal(o, op(q.contiguous(), cache, i64(lens)))
    check_decode(f64(o), None, f64(q), model, lens, [T, T], G)
    for n, m in (([150, 161], None), ([-1, 64], None), (lens, [3, 4]), (lens, [0, -1])):
        op(q, cache, i64(n), None if m is None else i64(m))
        assert csa.csa_check(op.ws) == 1
    op(q, cache, i64(lens), i64([0, 3]))
    assert csa.csa_check(op.ws) == 0


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
        cache, op, few = csa.KV8Cache(s, dev), csa.KV8Decode(s, dev), csa.KV8Sparse(s, dev, 1, n_first=0, n_last=1)
        with torch.cuda.stream(stream):
            cache.append(k, v, ln, ln)
            op(q, cache, ln)
            few(q, cache, ln)
        return cache, op, few
    _, op, few = run(torch.cuda.current_stream())
    want = op.o.clone(), few.o.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    cache, op, few = run(side)
    torch.cuda.synchronize()
    assert torch.equal(op.o, want[0]) and torch.equal(few.o, want[1])


def test_two_calls_at_once():
    # two objects on two streams, over one cache, many times over
    torch, csa, dev = _t()
    rng = np.random.default_rng(6)
    lens = [5000, 777, 3001]
    s, cache, _ = filled(rng, "bf16", 128, 2, lens, 5000, 8, step=4096)
    ln = i64(lens)
    calls = []
    for T in (1, 3):
        q = rows(rng, (3, T, 8, 128), "bf16")
        full, few = csa.KV8Decode(s, dev, T), csa.KV8Sparse(s, dev, 7, T)
        want = full(q, cache, ln).clone(), few(q, cache, ln).clone()
        calls.append((q, full, few, torch.cuda.Stream(dev), want))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, full, few, stream, _ in calls:
            full(q, cache, ln, stream=stream)
            few(q, cache, ln, stream=stream)
    torch.cuda.synchronize()
    for _, full, few, _, want in calls:
        assert torch.equal(full.o, want[0]) and torch.equal(few.o, want[1])


def test_offsets_past_32_bits():
    # arrays of more than 2^32 bytes: the last sequence's rows
    torch, csa, dev = _t()
    rng = np.random.default_rng(16)
    d, H, B, n_max = 128, 20, 2, 1 << 20      # K8: 5.4e9 bytes
    s = csa.make_shape(B, H, H, d, n_max, "bf16")
    cache, model = csa.KV8Cache(s, dev), Model(B, H, d)
    lens = append(cache, model, rng, "bf16", [0, 0], [3, 200], 200)
    q = rows(rng, (B, 1, H, d), "bf16")
    o = csa.KV8Decode(s, dev)(q, cache, i64(lens))
    check_decode(f64(o), None, f64(q), model, lens, [1, 1], 1)
    few = csa.KV8Sparse(s, dev, 3, n_first=1, n_last=1)
    few(q, cache, i64(lens))
    for h in range(H):
        ids, n = few.blocks[1, 0, h].tolist(), int(few.count[1, 0, h])
        span = np.stack([x[3] for x in model.blocks(1, h)])
        step = np.array([x[2][0] for x in model.blocks(1, h)])
        score = np.append(kv8.scores(float32(q)[1, 0, h:h + 1], span, step), 0)
        assert n == 3 and ids == kv8.choose(score, 3, 3, 1, 1)
        k, v = model.stands(1, h)
        pos = np.concatenate([np.arange(64 * j, min(64 * j + 64, 200)) for j in ids])
        check_row(f64(few.o)[1, 0, h], None, f64(q)[1, 0, h], k[pos], v[pos], h)
    K = torch.zeros(B, H, 130, d, dtype=torch.bfloat16, device=dev)
    V = torch.zeros_like(K)
    cache.unpack(K, V, i64(lens), i64([0, 60]))
    k, v = model.stands(1, H - 1)
    assert torch.equal(K[1, H - 1].cpu(), torch.from_numpy(k[60:190]).bfloat16())
    assert torch.equal(V[1, H - 1].cpu(), torch.from_numpy(v[60:190]).bfloat16())
    del cache
    # the last rows of a sequence of 2^20 tokens, in their far blocks
    s = csa.make_shape(1, 2, 2, d, n_max, "bf16")
    cache = csa.KV8Cache(s, dev)
    x = rows(rng, (1, 70, 2, d), "bf16")
    cache.append(x, x, i64([n_max]), i64([70]))
    K = torch.zeros(1, 2, 70, d, dtype=torch.bfloat16, device=dev)
    cache.unpack(K, K.clone(), i64([n_max]), i64([n_max - 70]))
    x = float32(x)[0, 6:, 1]
    want = torch.from_numpy(kv8.stands_for(kv8.codes(x, kv8.steps(x)), kv8.steps(x))).bfloat16()
    assert torch.equal(K[0, 1, 6:].cpu(), want)
