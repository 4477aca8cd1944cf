"""csa_kv4_decode on keys and values of very uneven sizes, against float64.

Each row's error is bounded by what that row attends to, not by the largest
key or value in sight.  With P_t the weights, mag_t the magnitude |m| + 15
Delta of a token's value and S_t = sum_c |q_c| (|m_c| + 15 Delta_c) / sqrt d
the one of its key's products (|v| and |k| in the incomplete block):
  * a score is off by eps_t <= (2^-21 + 8 sqrt(d) 2^-24) S_t: products to 22
    bits, d roundings of independent sign at eight standard deviations;
  * that moves the output o by sum_t P_t x_t (v_t - o) over the sum of the
    moved weights, x_t between +-(exp(eps_t) - 1): at most 2 sum_t P_t |x_t|
    max_c |v_t - o| while sum_t P_t |x_t| <= 1/2;
  * weights and sums over n tokens add (2^-20 + 8 sqrt(n) 2^-24) sum_t P_t
    mag_t.
The logarithm of the sum of weights is off by at most 2 sum_t P_t |x_t| + 2^-20
+ 8 sqrt(n) 2^-24, and its own roundings.
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


def stands(k, v):
    """What the cache of float32 rows k, v [n][d] stands for, and the
    magnitudes of its keys [n][d] and values [n]."""
    k, v = k.copy(), v.copy()
    magk, magv = np.abs(k).astype(np.float64), np.abs(v).max(1).astype(np.float64)
    w = len(k) // BLOCK * BLOCK
    if w:
        c, _, m, dl = quantize_keys(k[:w], w)
        m, dl = np.repeat(m, BLOCK, 0), np.repeat(dl, BLOCK, 0)
        k[:w] = kv4.stands_for(c, m, dl)
        magk[:w] = np.abs(m).astype(np.float64) + 15.0 * dl
        c, m, dl = kv4.quantize_values(v[:w])
        v[:w] = kv4.stands_for(c, m[:, None], dl[:, None])
        magv[:w] = np.abs(m).astype(np.float64) + 15.0 * dl
    return k, v, magk, magv


def decode(q, k, v, dtype):
    """Output [T][G][d] and lse [T][G] of the library for q [T][G][d], k, v
    [n][d], float32 arrays of values of the type."""
    import torch
    import certified_sparse_attention_gb300 as csa
    dev = torch.device("cuda:0")
    T, G, d = q.shape
    n = len(k)
    s = csa.make_shape(1, G, 1, d, n, dtype)
    cache = csa.KV4Cache(s, dev)
    el = torch.bfloat16 if dtype == "bf16" else torch.float32
    to = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev).to(el)
    ln = torch.tensor([n], dtype=torch.int64, device=dev)
    cache.append(to(k)[None, :, None], to(v)[None, :, None], ln)
    op = csa.KV4Decode(s, dev, T, with_lse=True)
    o = op(to(q)[None], cache, ln)
    assert csa.csa_check(op.ws) == 0
    return o[0].double().cpu().numpy(), op.lse[0].double().cpu().numpy()


def bf16(x):
    """float32 values rounded to bf16."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()


def check(q, k, v, dtype="f32"):
    """Every row within its own bound; returns the errors relative to the
    rows' sum_t P_t mag_t, and those of float32 attention."""
    o, lse = decode(q, k, v, dtype)
    T, G, d = q.shape
    n = len(k)
    ks, vs, magk, magv = stands(k, v)
    mine, plain = [], []
    for t in range(T):
        seen = n - T + t + 1
        for h in range(G):
            x = q[t, h].astype(np.float64)
            s = ks[:seen].astype(np.float64) @ x / np.sqrt(d)
            p = np.exp(s - s.max())
            p /= p.sum()
            ref = p @ vs[:seen].astype(np.float64)
            S = magk[:seen] @ np.abs(x) / np.sqrt(d)
            with np.errstate(over="ignore"):
                e = np.expm1((2.0 ** -21 + 8 * np.sqrt(d) * 2.0 ** -24) * S)
            e = np.where(p == 0, 0.0, e)
            A = p @ magv[:seen]
            assert p @ e <= 0.5
            away = np.abs(vs[:seen].astype(np.float64) - ref).max(1)
            lim = 2 * (p @ (e * away)) + \
                (2.0 ** -20 + 8 * np.sqrt(seen) * 2.0 ** -24) * A
            err = np.abs(o[t, h] - ref).max()
            assert err <= lim, (t, h, err / A, lim / A)
            ls = s.max() + np.log(np.exp(s - s.max()).sum())
            lim = 2 * (p @ e) + 2.0 ** -20 + 8 * np.sqrt(seen) * 2.0 ** -24 + 2.0 ** -22 * abs(ls)
            assert abs(lse[t, h] - ls) <= lim, (t, h, lse[t, h], ls, lim)
            mine.append(err / A)
            s = (ks[:seen] @ q[t, h]) / np.float32(np.sqrt(d))
            p = np.exp(s - s.max())
            plain.append(np.abs((p / p.sum()) @ vs[:seen] - ref).max() / A)
    return max(mine), max(plain)


SHAPES = [(4, 1), (8, 1), (4, 3), (8, 8)]      # G, T: tiles of 4 and of 8 rows, 1 to 8 of them


def case(rng, G, T, d, n):
    """Queries around u = (+-1)_c, keys and values around 0."""
    u = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    q = (u + 0.1 * rng.normal(size=(T, G, d))).astype(np.float32)
    k = (0.1 * rng.normal(size=(n, d))).astype(np.float32)
    v = rng.normal(size=(n, d)).astype(np.float32)
    return u, q, k, v


@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 16, 2.0 ** 20])
@pytest.mark.parametrize("large,at", [(3, 9), (3, 64 * 12 + 1), (64 * 11 + 5, 64 * 11 + 40),
                                      (64 * 23 + 60, 64 * 23 + 2), (64 * 23 + 60, 0)])
def test_values_of_tokens_that_do_not_count(G, T, d, ratio, large, at):
    # every row attends to one token; another one, at a weight of e^-40, has
    # values larger by the ratio: in the first, a later and the last whole
    # block, the two in one block and apart
    rng = np.random.default_rng([G, T, d, at])
    u, q, k, v = case(rng, G, T, d, 64 * 24 + 7)
    k[at] = (20.0 / np.sqrt(d)) * u
    k[large] = -k[at]
    v[large] *= ratio
    check(q, k, v)


@pytest.mark.parametrize("G,T", SHAPES)
def test_values_shrink_and_grow_along_the_sequence(G, T):
    # every block's values 2^6 smaller than the one's before (then larger),
    # while the scores rise (fall) by as much, so that all of them count
    rng = np.random.default_rng([G, T])
    d, n = 64, 64 * 16 + 3
    u, q, k, v = case(rng, G, T, d, n)
    step = np.minimum(np.arange(n) // BLOCK, 15) - 7.5
    for sign in (1.0, -1.0):
        kk = k + (sign * step[:, None] * 6 * np.log(2.0) / np.sqrt(d)) * u
        vv = v * (2.0 ** (-6 * sign * step))[:, None]
        check(q, kk.astype(np.float32), vv.astype(np.float32))


@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** -98, 2.0 ** -40, 2.0 ** 40, 2.0 ** 96])
def test_values_of_one_size_that_jump_once(G, T, scale):
    # constant rows (no step) in the first blocks, then values of any size
    rng = np.random.default_rng([G, T, 5])
    d, n = 64, 64 * 20
    _, q, k, v = case(rng, G, T, d, n)
    v *= np.float32(scale)
    v[:64 * 13] = np.float32(0.5 * scale)
    check(q, k, v)


@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [True, False])
def test_keys_large_where_the_query_is_small(G, T, d, first):
    # a channel of keys around 2^30 against a query of 2^-30 there, or of 0,
    # in the first block only or in all of them
    rng = np.random.default_rng([G, T, d])
    n = 64 * 15 + 9
    for small in (2.0 ** -30, 0.0):
        _, q, k, v = case(rng, G, T, d, n)
        k *= 8
        k[:64 if first else n, 5] *= np.float32(2.0 ** 30)
        q[..., 5] = small
        check(q, k, v)


@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -24, 2.0 ** -9, 2.0 ** 9, 2.0 ** 24, 2.0 ** 60])
def test_keys_of_any_size_with_channels_of_zeros(G, T, scale):
    # heads padded with zeros (whose step is 1), queries that make up for the
    # size of the keys; keys that get smaller on the way
    rng = np.random.default_rng([G, T, 3])
    d, n = 64, 64 * 15
    for shrink in (1.0, 2.0 ** -20):
        _, q, k, v = case(rng, G, T, d, n)
        k *= 8 * scale
        k[64 * 7:] *= shrink
        q /= scale
        k[:, 40:] = 0
        q[..., 40:] = 0
        check(q, k.astype(np.float32), v)


def test_queries_of_very_different_sizes_share_a_tile():
    # rows of one tile from 2^-40 to 2^40, and rows of zeros
    rng = np.random.default_rng(3)
    for G, T in SHAPES:
        _, q, k, v = case(rng, G, T, 64, 64 * 9 + 2)
        k *= np.float32(2.0 ** -40)
        q *= (2.0 ** np.linspace(-40, 40, T * G)).reshape(T, G, 1).astype(np.float32)
        q[0, G // 2] = 0
        check(q, k, v)


@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("low", [2.0 ** 10, 2.0 ** 14, 2.0 ** 18])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_after_blocks_of_very_low_ones(G, T, low, d):
    # the first half of the blocks score about -low throughout; the two tokens
    # that every row attends to (one code apart) lie in one block after them
    rng = np.random.default_rng([G, T, d])
    u, q, k, v = case(rng, G, T, d, 64 * 23 + 7)
    k[:64 * 12] -= ((low / np.sqrt(d)) * u).astype(np.float32)
    k[64 * 13 + 3] = (20.0 / np.sqrt(d)) * u
    k[64 * 13 + 40] = (18.6 / np.sqrt(d)) * u
    check(q, k, v)


def test_errors_next_to_those_of_float32_attention():
    # operands in two halves keep 22 bits for 24, and matrix instructions
    # truncate where float32 rounds: four times two
    rng = np.random.default_rng(40)
    mine = plain = 0.0
    for _ in range(12):
        G, T = SHAPES[rng.integers(len(SHAPES))]
        d, n = int(rng.choice([64, 128])), int(rng.integers(64, 3000))
        _, q, k, v = case(rng, G, T, d, n)
        a, b = check(q, 8 * k, v)
        mine, plain = mine + a, plain + b
    assert mine <= 8 * plain, mine / plain


@pytest.mark.parametrize("G,T", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_uneven_bf16(G, T, d):
    # large values at no weight, a channel of large keys where the query is
    # 0, and low blocks first, together, in 16 bits
    rng = np.random.default_rng([G, T, d, 16])
    u, q, k, v = case(rng, G, T, d, 64 * 22 + 30)
    q[..., 7] = u[7] = 0.0
    k[:64 * 11] -= ((2.0 ** 12 / np.sqrt(d)) * u).astype(np.float32)
    k[64 * 15 + 8] = (20.0 / np.sqrt(d)) * u
    k[64 * 15 + 44] = (18.0 / np.sqrt(d)) * u
    k[::5, 7] *= 2.0 ** 24
    k[64 * 15 + 50] = -k[64 * 15 + 8]
    v[64 * 15 + 50] *= 2.0 ** 18
    check(bf16(q), bf16(k), bf16(v), "bf16")
