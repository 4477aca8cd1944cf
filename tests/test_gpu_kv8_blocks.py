"""Blocks chosen by a cheap score (csa_kv8_select) and the attention over listed
blocks (csa_kv8_decode_blocks), on the GPU: choices against oracle/kv8.py,
number for number; attention within the tolerances of test_gpu_kv8.py."""
import numpy as np
import pytest

from oracle import kv8
from tests.test_gpu_kv8 import (BLOCK, Model, _lib, _t, append, check_row, f64, filled,  # noqa: F401
                                float32, i64, on_gpu, rows, spoil, tdtype)

pytestmark = pytest.mark.gpu


def i32(x):
    torch, _, dev = _t()
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def chosen(model, q, b, g, n, m, t, n_sel, n_first, n_last):
    """The oracle's list for one token; q [G, d]."""
    pos = n - m + t
    if pos < 0:
        return []
    own = pos // BLOCK
    blocks = model.blocks(b, g)[:own]
    score = np.zeros(own + 1, np.float32)
    if blocks:
        score[:len(blocks)] = kv8.scores(q, np.stack([x[3] for x in blocks]), np.array([x[2][0] for x in blocks]))
    return kv8.choose(score, own, n_sel, n_first, n_last)


def check_choice(op, q, model, lens, nq):
    """blocks and count of every row; rows past nq are 77."""
    blocks, count = op.blocks.cpu().numpy(), op.count.cpu().numpy()
    B, T, H, N = blocks.shape
    G = q.shape[2] // H
    qn = float32(q)
    for b in range(B):
        for t in range(T):
            for g in range(H):
                if t >= nq[b]:
                    assert np.all(blocks[b, t, g] == 77) and count[b, t, g] == 77
                    continue
                want = chosen(model, qn[b, t, g * G:(g + 1) * G], b, g, lens[b], nq[b], t, N, op.n_first, op.n_last)
                assert count[b, t, g] == len(want)
                assert blocks[b, t, g].tolist() == want + [-1] * (N - len(want)), (b, t, g)


def check_listed(o, lse, q, model, lens, nq, blocks, count):
    """Rows t < nq over the listed blocks."""
    B, T, Hq, d = o.shape
    H = blocks.shape[2]
    G = Hq // H
    for b in range(B):
        for g in range(H):
            k, v = model.stands(b, g)
            for t in range(nq[b]):
                seen = max(0, lens[b] - nq[b] + t + 1)
                ids = blocks[b, t, g, :count[b, t, g]]
                pos = np.array([p for j in ids for p in range(64 * j, 64 * j + 64) if p < seen], int)
                for h in range(g * G, (g + 1) * G):
                    check_row(o[b, t, h], lse[b, t, h], q[b, t, h], k[pos], v[pos], (b, t, h))


@pytest.mark.parametrize("G,T,N,first,last", [
    (1, 1, 1, 0, 1), (4, 1, 5, 1, 2), (8, 1, 16, 2, 4), (2, 3, 6, 0, 1), (4, 5, 9, 1, 1), (1, 16, 4, 2, 2),
    (8, 8, 3, 1, 1), (4, 16, 40, 1, 2), (2, 2, 200, 1, 2)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("f32", 128), ("bf16", 64)])
def test_choice_and_attention(G, T, N, first, last, dtype, d):
    torch, csa, dev = _t()
    rng = np.random.default_rng(100 * G + T + d)
    H = 2
    lens = [0, 1, 64, 65, 333, 1311, 2112, 2111]
    nq = [int(rng.integers(0, T + 1)) for _ in lens] if T > 1 else [1] * len(lens)
    nq[1], nq[6] = T, T
    s, cache, model = filled(rng, dtype, d, H, lens, 2200, G * H, step=1024)
    q = rows(rng, (len(lens), T, G * H, d), dtype)
    q[2] *= 0.05
    op = csa.KV8Sparse(s, dev, N, T, first, last, with_lse=True)
    op.blocks.fill_(77)
    op.count.fill_(77)
    op.ws.fill_(0xFF)
    op.o.fill_(55.0)
    o = op(q, cache, i64(lens), i64(nq))
    assert csa.csa_check(op.status) == 0 and csa.csa_check(op.ws) == 0
    check_choice(op, q, model, lens, nq)
    check_listed(f64(o), f64(op.lse), f64(q), model, lens, nq, op.blocks.cpu().numpy(), op.count.cpu().numpy())
    for b in range(len(lens)):
        assert bool((o[b, nq[b]:] == 55.0).all())
    # again: the same bits
    first_o, first_b = o.clone(), op.blocks.clone()
    op(q, cache, i64(lens), i64(nq))
    assert torch.equal(first_o, op.o) and torch.equal(first_b, op.blocks)


def test_all_blocks_listed_is_the_whole_cache():
    torch, csa, dev = _t()
    rng = np.random.default_rng(3)
    lens = [700, 64, 3000]
    s, cache, model = filled(rng, "bf16", 128, 2, lens, 3000, 8, step=1024)
    q = rows(rng, (3, 2, 8, 128), "bf16")
    few, full = csa.KV8Sparse(s, dev, 47, 2, with_lse=True), csa.KV8Decode(s, dev, 2, with_lse=True)
    few(q, cache, i64(lens))
    full(q, cache, i64(lens))
    check_listed(f64(few.o), f64(few.lse), f64(q), model, lens, [2] * 3, few.blocks.cpu().numpy(), few.count.cpu().numpy())
    assert few.count[2].unique().tolist() == [47] and few.count[1].unique().tolist() == [1]
    # two orders of the same sums
    assert float((few.o - full.o).abs().max()) <= 2.0 ** -17 * max(float(x.abs().max()) for x in (few.o, full.o)) * 8


def with_spans(s, span, scale):
    """A cache of given spans and steps of the keys, and zeros otherwise."""
    torch, csa, dev = _t()
    cache = csa.KV8Cache(s, dev)
    cache.span.copy_(torch.from_numpy(span).to(dev))
    cache.scale[..., 0].copy_(torch.from_numpy(scale).to(dev))
    return cache


def spans_choice(s, cache, q, lens, N, first, last, T=1):
    torch, csa, dev = _t()
    op = csa.KV8Sparse(s, dev, N, T, first, last)
    op.select(q, cache, i64(lens))
    assert csa.csa_check(op.status) == 0
    return op.blocks.cpu().numpy(), op.count.cpu().numpy()


@pytest.mark.parametrize("B,H,G,T,n,N", [
    (1, 1, 4, 1, 64 * 3000, 100), (1, 2, 1, 16, 64 * 700 + 5, 33), (3, 16, 8, 1, 64 * 130 + 1, 7),
    (40, 8, 2, 2, 64 * 65, 5), (1, 1, 8, 2, 64 * 513, 512), (2, 1, 4, 16, 64 * 9000 + 63, 1024)])
def test_choice_over_many_blocks(B, H, G, T, n, N):
    # random codes and steps, among them many equal scores; clusters of one CTA
    # to eight, one and more clusters to a sequence and head
    torch, csa, dev = _t()
    rng = np.random.default_rng(n)
    d = 64
    s = csa.make_shape(B, H * G, H, d, n, "bf16")
    nblk = -(-n // BLOCK)
    span = rng.integers(1, 256, (B, H, nblk, 2, d)).astype(np.uint8)
    span[:, :, nblk // 3:nblk // 2] = span[:, :, :1]              # ties
    span[:, :, 1::5, 1:] = span[:, :, 1:2, 1:]
    scale = (0.01 * 2.0 ** rng.integers(-2, 3, (B, H, nblk))).astype(np.float32)
    scale[:, :, nblk // 3:nblk // 2] = 0.01
    cache = with_spans(s, span, scale)
    q = rows(rng, (B, T, H * G, d), "bf16")
    lens = [n - 100 * (b % 3) for b in range(B)]
    got, count = spans_choice(s, cache, q, lens, N, 1, 2, T)
    qn = float32(q)
    for b in range(0, B, 7):
        for t in range(T):
            for g in range(0, H, 5):
                own = (lens[b] - T + t) // BLOCK
                score = np.append(kv8.scores(qn[b, t, g * G:(g + 1) * G], span[b, g, :own], scale[b, g, :own]), 0)
                want = kv8.choose(score, own, N, 1, 2)
                assert got[b, t, g].tolist() == want + [-1] * (N - len(want)) and count[b, t, g] == len(want)


def test_choice_of_equal_and_special_scores():
    torch, csa, dev = _t()
    d, n, N = 128, 64 * 50, 8
    s = csa.make_shape(1, 2, 1, d, n, "f32")
    rng = np.random.default_rng(2)
    q = rng.normal(size=(1, 1, 2, d)).astype(np.float32)
    q[..., 3] = np.abs(q[..., 3]) + 0.5
    flat = np.full((1, 1, 50, 2, d), 128, np.uint8)
    ones = np.full((1, 1, 50), 0.5, np.float32)
    run = lambda span, scale, q=q: spans_choice(s, with_spans(s, span, scale), on_gpu(q), [n], N, 1, 2)[0][0, 0, 0].tolist()
    # no score differs: the lowest numbers
    assert run(flat, ones) == [0, 1, 2, 3, 4, 5, 48, 49]
    # a query of zeros: the same, whatever the spans
    assert run(rng.integers(1, 256, flat.shape).astype(np.uint8), ones, 0 * q) == [0, 1, 2, 3, 4, 5, 48, 49]
    # one better block, one worse one
    up = flat.copy()
    up[0, 0, 30, 0, 3], up[0, 0, 2, :, 3] = 129, 127
    assert run(up, ones) == [0, 1, 3, 4, 5, 30, 48, 49]
    # a NaN or infinite step (a block that holds one) is not passed over: 0 times
    # infinity is a NaN as well
    for bad in (np.nan, np.inf):
        scale = ones.copy()
        scale[0, 0, 33] = bad
        assert run(up, scale) == [0, 1, 3, 4, 30, 33, 48, 49]
    # products that overflow: +infinity above, -infinity below
    big = up.copy()
    scale = np.full_like(ones, 3e38)
    got = run(big, scale, q * np.float32(1e30))
    assert 30 in got and 2 not in got
    # a NaN in a query: every score is one, the lowest numbers
    bad = q.copy()
    bad[0, 0, 1, 7] = np.nan
    assert run(up, ones, bad) == [0, 1, 2, 3, 4, 5, 48, 49]


def test_choice_refuses_lengths():
    torch, csa, dev = _t()
    s = csa.make_shape(3, 2, 1, 64, 640, "bf16")
    cache = csa.KV8Cache(s, dev)
    q = torch.ones(3, 2, 2, 64, dtype=torch.bfloat16, device=dev)
    op = csa.KV8Sparse(s, dev, 3, 2)
    for lens, nq in (([641, 640, 5], [2, 2, 2]), ([-1, 640, 5], [2, 2, 2]), ([5, 640, 5], [3, 1, 2]), ([5, 640, 5], [-1, 1, 2])):
        op.blocks.fill_(77)
        op.count.fill_(77)
        op.select(q, cache, i64(lens), i64(nq))
        assert csa.csa_check(op.status) == 1
        assert bool((op.blocks[0] == 77).all()) and bool((op.count[0] == 77).all())
        assert op.blocks[1, 0, 0].tolist() == [0, 8, 9] and op.blocks[2, 0, 0].tolist() == [0, -1, -1]
    op.select(q, cache, i64([0, 640, 1]))
    assert csa.csa_check(op.status) == 0 and op.count[:, :, 0].tolist() == [[0, 0], [3, 3], [0, 1]]


def test_lists_of_the_caller():
    # any ascending lists; an empty one; the token's own block alone or left out;
    # rows whose list is none are NaN and the others as they would be
    torch, csa, dev = _t()
    rng = np.random.default_rng(8)
    T, H, G, d, n = 3, 2, 2, 128, 64 * 11 + 1
    lens, nq = [n, 64 * 10, 700], [3, 3, 2]
    s, cache, model = filled(rng, "bf16", d, H, lens, n, H * G)
    q = rows(rng, (3, T, H * G, d), "bf16")
    op = csa.KV8Sparse(s, dev, 6, T, with_lse=True)
    lists = [[[[0, 2, 5], [11]], [[], [10]], [[3, 4, 5, 6, 7, 11], [0]]],
             [[[9], [8, 9]], [[0, 9], [1]], [[2, 3, 9], [0, 1, 2, 3, 4, 9]]],
             [[[10], [0, 10]], [[0], [5, 6, 9]], [[0], [0]]]]
    # (positions of sequence 0: 702, 703, 704; block 11 begins at 704)
    lists[0][0][1], lists[0][1][1] = [10], [4, 10]
    blocks = np.full((3, T, H, 6), -1)
    count = np.zeros((3, T, H), int)
    for b in range(3):
        for t in range(T):
            for g in range(H):
                blocks[b, t, g, :len(lists[b][t][g])] = lists[b][t][g]
                count[b, t, g] = len(lists[b][t][g])
    op.ws.fill_(0xFF)
    o = op.attend(q, cache, i64(lens), i64(nq), i32(blocks), i32(count))
    assert csa.csa_check(op.ws) == 0
    check_listed(f64(o), f64(op.lse), f64(q), model, lens, nq, blocks, count)
    good, lse = o.clone(), op.lse.clone()
    bad = blocks.copy()
    cnt = count.copy()
    bad[0, 0, 0, :3] = [0, 5, 2]          # not ascending
    bad[0, 2, 0, :6] = [3, 4, 4, 6, 7, 11]     # one twice
    bad[0, 0, 1, 0] = 11                  # past the token's own
    bad[1, 0, 0, 0] = -1                  # below zero
    bad[1, 1, 0, :2] = [0, 1 << 30]
    cnt[1, 2, 0], cnt[2, 0, 0] = 7, -1
    broken = [(0, 0, 0), (0, 2, 0), (0, 0, 1), (1, 0, 0), (1, 1, 0), (1, 2, 0), (2, 0, 0)]
    o = op.attend(q, cache, i64(lens), i64(nq), i32(bad), i32(cnt))
    for b in range(3):
        for t in range(nq[b]):
            for g in range(H):
                row = slice(g * G, (g + 1) * G)
                if (b, t, g) in broken:
                    assert torch.isnan(o[b, t, row]).all() and torch.isnan(op.lse[b, t, row]).all()
                else:
                    assert torch.equal(o[b, t, row], good[b, t, row]) and torch.equal(op.lse[b, t, row], lse[b, t, row])


@pytest.mark.parametrize("G,T,N", [(4, 1, 150), (8, 2, 300), (1, 16, 64), (4, 1, 250), (2, 16, 290)])
def test_lists_cut_over_ctas(G, T, N):
    # long lists of few rows, cut or shared by a few CTAs, refused ones among them
    torch, csa, dev = _t()
    rng = np.random.default_rng(G)
    d, lens = 64, [64 * 300 + 17, 64 * 290]
    s, cache, model = filled(rng, "f32", d, 1, lens, lens[0], G, step=8192)
    q = rows(rng, (2, T, G, d), "f32")
    op = csa.KV8Sparse(s, dev, N, T, with_lse=True)
    blocks = np.full((2, T, 1, N), -1)
    count = np.zeros((2, T, 1), int)
    for b in range(2):
        for t in range(T):
            m = int(rng.integers(0, min(N, 280)))
            ids = np.sort(rng.permutation(285)[:m])
            if t % 2 == 0 and m < N:
                ids = np.append(ids, (lens[b] - T + t) // BLOCK)
            blocks[b, t, 0, :len(ids)], count[b, t, 0] = ids, len(ids)
    op.ws.fill_(0xFF)
    o = op.attend(q, cache, i64(lens), None, i32(blocks), i32(count))
    assert csa.csa_check(op.ws) == 0
    check_listed(f64(o), f64(op.lse), f64(q), model, lens, [T, T], blocks, count)
    assert bool(torch.isfinite(o).all())
    if count[1, 0, 0] < 2:
        count[1, 0, 0] = 2
    blocks[1, 0, 0, :2] = [5, 5]
    o2 = op.attend(q, cache, i64(lens), None, i32(blocks), i32(count))
    assert torch.isnan(o2[1, 0]).all() and torch.isnan(op.lse[1, 0]).all() and torch.equal(o2[0], o[0])


def test_no_query_token_at_all():
    torch, csa, dev = _t()
    rng = np.random.default_rng(1)
    for n in (500, 5000):
        s, cache, _ = filled(rng, "bf16", 64, 1, [n, n], n, 2, step=4096)
        q = rows(rng, (2, 2, 2, 64), "bf16")
        op = csa.KV8Sparse(s, dev, 40, 2)
        op.o.fill_(55.0)
        op(q, cache, i64([n, n]), i64([0, 0]))
        assert csa.csa_check(op.ws) == 0 and bool((op.o == 55.0).all())
        op(q, cache, i64([n, n]), i64([0, 2]))
        assert bool((op.o[0] == 55.0).all()) and not bool((op.o[1] == 55.0).any())


@pytest.mark.parametrize("n", [700, 6000])
def test_a_layer_decoded_with_one_graph(n):
    # rotation, append, choice, attention over the chosen blocks and over all,
    # captured once and replayed token by token, lengths on the device
    torch, csa, dev = _t()
    rng = np.random.default_rng(21)
    B, Hq, H, d, steps, N = 2, 8, 2, 128, 5, 6
    n_max = n + 10
    s = csa.make_shape(B, Hq, H, d, n_max, "bf16")
    start = [n, n // 64 * 64 - 3]                # a block fills on the way
    f = 500000.0 ** (-np.arange(d // 2) / (d // 2))
    rope, cache, model = csa.QKNormRope(s, dev, inv_freq=f), csa.KV8Cache(s, dev), Model(B, H, d)
    full, few = csa.KV8Decode(s, dev), csa.KV8Sparse(s, dev, N, with_lse=True)
    k, v = rows(rng, (B, n, H, d), "bf16"), rows(rng, (B, n, H, d), "bf16")
    lens = i64(start)
    cache.append(k, v, lens, lens)
    model.add(float32(k), float32(v), start)
    x = torch.zeros(B, 1, Hq + 2 * H, d, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(B, 1, Hq, d, dtype=torch.bfloat16, device=dev)
    k, v = torch.zeros(B, 1, H, d, dtype=torch.bfloat16, device=dev), torch.zeros(B, 1, H, d, dtype=torch.bfloat16, device=dev)

    def token():
        rope(x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:], k, v, lens, to_cache=False, q_out=q)
        cache.append(k, v, lens)
        few(q, cache, lens)
        full(q, cache, lens)

    side, graph = torch.cuda.Stream(dev), None
    torch.cuda.synchronize()
    for t in range(steps):
        lens += 1
        x.copy_(rows(rng, tuple(x.shape), "bf16"))
        torch.cuda.synchronize()
        if t == 0:
            with torch.cuda.stream(side):
                token()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    token()
            graph.replay()
        torch.cuda.synchronize()
        now = [a + t + 1 for a in start]
        model.add(float32(k), float32(v), [1] * B)
        for word in (few.ws, few.status, full.ws, cache.status, cache.refused):
            assert csa.csa_check(word) == 0
        check_choice(few, q, model, now, [1] * B)
        check_listed(f64(few.o), f64(few.lse), f64(q), model, now, [1] * B, few.blocks.cpu().numpy(), few.count.cpu().numpy())
        for b in range(B):
            for h in range(Hq):
                kk, vv = model.stands(b, h // (Hq // H))
                check_row(f64(full.o)[b, 0, h], None, f64(q)[b, 0, h], kk, vv, (b, h))


def test_choice_at_the_longest_context():
    # CSA_KV8_MAX_SELECT_TOKENS tokens, several query tokens
    torch, csa, dev = _t()
    n, T, d, N = 3 << 20, 3, 64, 20
    s = csa.make_shape(1, 2, 1, d, n, "bf16")
    rng = np.random.default_rng(3)
    nblk = n // BLOCK
    span = rng.integers(1, 256, (1, 1, nblk, 2, d)).astype(np.uint8)
    scale = np.full((1, 1, nblk), 0.02, np.float32)
    q = rows(rng, (1, T, 2, d), "bf16")
    got, count = spans_choice(s, with_spans(s, span, scale), q, [n], N, 1, 2, T)
    for t in range(T):
        own = (n - T + t) // BLOCK
        score = np.append(kv8.scores(float32(q)[0, t], span[0, 0, :own], scale[0, 0, :own]), 0)
        assert got[0, t, 0].tolist() == kv8.choose(score, own, N, 1, 2) and count[0, t, 0] == N


@pytest.mark.parametrize("T,N", [(2, 121), (4, 300), (8, 200)])
def test_workspace_for_more_tokens_serves_fewer(T, N):
    # lists of T tokens are shared by CTAs, of one token cut and joined from the
    # workspace, which was sized for T
    torch, csa, dev = _t()
    rng = np.random.default_rng(N)
    B, H, G, d, n = 2, 8, 1, 64, 64 * 310 + 5
    s, cache, model = filled(rng, "bf16", d, H, [n, n - 70], n, H * G, step=8192)
    q = rows(rng, (B, 1, H * G, d), "bf16")
    op = csa.KV8Sparse(s, dev, N, with_lse=True)
    op(q, cache, i64([n, n - 70]))
    want = op.o.clone()
    check_listed(f64(op.o), f64(op.lse), f64(q), model, [n, n - 70], [1, 1], op.blocks.cpu().numpy(), op.count.cpu().numpy())
    size = csa.csa_kv8_workspace_size(s, T, N)
    assert size >= csa.csa_kv8_workspace_size(s, 1, N) and size >= csa.csa_kv8_workspace_size(s, T, N - 7)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    op.o.fill_(55.0)
    assert csa.csa_kv8_decode_blocks(s, cache.desc, 1, q, q, i64([n, n - 70]), None, op.blocks, op.count, N,
                                     op.o, None, ws, size) == 0
    assert csa.csa_check(ws) == 0 and torch.equal(op.o, want)


@pytest.mark.parametrize("dtype,d,B,H,G,T,n,N", [
    ("bf16", 128, 1, 2, 4, 1, 64 * 4096 + 5, 16), ("f32", 64, 1, 1, 2, 5, 64 * 4096 + 5, 300),
    ("bf16", 64, 2, 1, 8, 1, 64 * 5003, 1024), ("f32", 128, 1, 1, 1, 16, 64 * 4100 + 3, 7),
    ("bf16", 128, 1, 1, 1, 1, 64 * 16384, 256), ("f32", 128, 1, 1, 4, 2, 64 * 16384 - 1, 1024),
    ("f32", 64, 1, 2, 8, 1, 64 * 16384 + 63, 1), ("bf16", 128, 1, 1, 4, 1, 64 * 36864, 64)])
def test_choice_by_sixteen_warps(dtype, d, B, H, G, T, n, N):
    # contexts of 4096 blocks and more, few enough rows for half of the SMs: chunks of
    # 256 blocks, one token's scores to a CTA; many equal scores
    torch, csa, dev = _t()
    rng = np.random.default_rng(n + d)
    s = csa.make_shape(B, H * G, H, d, n, dtype)
    nblk = -(-n // BLOCK)
    span = rng.integers(1, 256, (B, H, nblk, 2, d)).astype(np.uint8)
    span[:, :, nblk // 3:nblk // 2] = span[:, :, :1]
    scale = (0.01 * 2.0 ** rng.integers(-2, 3, (B, H, nblk))).astype(np.float32)
    scale[:, :, nblk // 3:nblk // 2] = 0.04
    q = rows(rng, (B, T, H * G, d), dtype)
    lens = [n - 64 * 300 * b for b in range(B)]
    first, last = (0, 1) if N == 1 else (1, 2)
    got, count = spans_choice(s, with_spans(s, span, scale), q, lens, N, first, last, T)
    qn = float32(q)
    for b in range(B):
        for t in range(T):
            for g in range(H):
                own = (lens[b] - T + t) // BLOCK
                score = np.append(kv8.scores(qn[b, t, g * G:(g + 1) * G], span[b, g, :own], scale[b, g, :own]), 0)
                assert got[b, t, g].tolist() == kv8.choose(score, own, N, first, last), (b, t, g)
                assert count[b, t, g] == N


@pytest.mark.parametrize("T,n", [(1, 3 << 20), (2, (3 << 20) - 64)])
def test_choice_at_the_longest_context_of_wide_heads(T, n):
    # d = 128 near CSA_KV8_MAX_SELECT_TOKENS: beside the scores there is room for one
    # chunk of 64 blocks
    torch, csa, dev = _t()
    d, N = 128, 20
    s = csa.make_shape(1, 4, 1, d, 3 << 20, "bf16")
    rng = np.random.default_rng(T)
    nblk = (3 << 20) // BLOCK
    span = rng.integers(1, 256, (1, 1, nblk, 2, d)).astype(np.uint8)
    span[:, :, 1000:9000] = span[:, :, :1]
    scale = np.full((1, 1, nblk), 0.02, np.float32)
    q = rows(rng, (1, T, 4, d), "bf16")
    got, count = spans_choice(s, with_spans(s, span, scale), q, [n], N, 1, 2, T)
    for t in range(T):
        own = (n - T + t) // BLOCK
        score = np.append(kv8.scores(float32(q)[0, t], span[0, 0, :own], scale[0, 0, :own]), 0)
        assert got[0, t, 0].tolist() == kv8.choose(score, own, N, 1, 2) and count[0, t, 0] == N


@pytest.mark.parametrize("N", [320, 400])
def test_long_runs_of_lists(N):
    # more listed blocks of an item to one CTA than it holds numbers of: shared by two
    # CTAs (320), and cut into runs of about 170 (400)
    torch, csa, dev = _t()
    rng = np.random.default_rng(N)
    T, H, d, n = 16, 4, 64, 64 * 420 + 17
    s, cache, model = filled(rng, "bf16", d, H, [n], n, H, step=8192)
    q = rows(rng, (1, T, H, d), "bf16")
    q[0, 3] *= 0.02
    op = csa.KV8Sparse(s, dev, N, T, with_lse=True)
    blocks = np.full((1, T, H, N), -1)
    count = rng.integers(N - 30, N + 1, (1, T, H))
    count[0, 0, 0], count[0, 5, 1] = N, 129
    for t in range(T):
        for g in range(H):
            m = count[0, t, g]
            own = (n - T + t) // BLOCK
            ids = np.sort(rng.permutation(own)[:m])
            if (t + g) % 2:
                ids[-1] = own
            blocks[0, t, g, :m] = ids
    op.ws.fill_(0xFF)
    o = op.attend(q, cache, i64([n]), None, i32(blocks), i32(count))
    assert csa.csa_check(op.ws) == 0
    check_listed(f64(o), f64(op.lse), f64(q), model, [n], [T], blocks, count)
