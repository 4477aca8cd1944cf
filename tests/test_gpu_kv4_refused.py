"""An append's refusal outlives the calls after it (KV4Cache.refused)."""
import pytest

from tests.gpu_common import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _cache(B, n_max, T):
    import torch
    import certified_sparse_attention_gb300 as csa
    dev = torch.device("cuda:0")
    s = csa.make_shape(B, 1, 1, 64, n_max, "bf16")
    x = torch.ones(B, T, 1, 64, dtype=torch.bfloat16, device=dev)
    out = torch.zeros(B, 1, n_max, 64, dtype=torch.bfloat16, device=dev)

    def i64(*v):
        return torch.tensor(v, dtype=torch.int64, device=dev)
    return torch, csa, csa.KV4Cache(s, dev), x, out, i64


@pytest.mark.parametrize("lens,new", [((101, 70), (70, 70)), ((70, 69), (70, 70)),
                                      ((71, 70), (71, 70)), ((70, 70), (70, -1))])
def test_refused_append_then_good_calls(lens, new):
    torch, csa, cache, x, out, i64 = _cache(2, 100, 70)
    good = i64(70, 70)
    cache.append(x, x, good)
    cache.unpack(out, out.clone(), good)
    assert csa.csa_check(cache.refused) == csa.CSA_OK
    cache.append(x, x, i64(*lens), i64(*new))
    cache.unpack(out, out.clone(), good)
    assert csa.csa_check(cache.status) == csa.CSA_OK        # the last call's
    assert csa.csa_check(cache.refused) == 1
    cache.append(x, x, good)
    assert csa.csa_check(cache.status) == csa.CSA_OK
    assert csa.csa_check(cache.refused) == 1
    cache.refused.zero_()
    cache.append(x, x, good)
    assert csa.csa_check(cache.refused) == csa.CSA_OK
    # an unpack out of range leaves the word alone: nothing of the cache is lost
    cache.unpack(out, out.clone(), i64(101, 70))
    assert csa.csa_check(cache.status) == 1
    assert csa.csa_check(cache.refused) == csa.CSA_OK


def test_refused_append_within_a_graph():
    # three tokens to a graph: a sequence is full before the last of them
    torch, csa, cache, x, out, i64 = _cache(2, 100, 1)
    lens, one = i64(97, 10), i64(1, 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        cache.append(x, x, lens, one)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for _ in range(2):
            lens += 1
            cache.append(x, x, lens, one)
        cache.unpack(out, out, torch.clamp(lens, max=100))
    g.replay()
    torch.cuda.synchronize()
    assert csa.csa_check(cache.refused) == csa.CSA_OK
    g.replay()
    torch.cuda.synchronize()
    assert csa.csa_check(cache.status) == csa.CSA_OK
    assert csa.csa_check(cache.refused) == 1


def test_append_without_a_word_for_its_status():
    # a C caller may give either word, both or none
    import ctypes
    torch, csa, cache, x, out, i64 = _cache(2, 100, 70)
    bad = i64(101, 70)
    st = ctypes.byref(csa.csa_strides(*x.stride()[:3]))
    call = csa.load_library().csa_kv4_append
    none = csa.csa_kv4(*[getattr(cache.desc, f) for f, _ in csa.csa_kv4._fields_[:6]])
    for desc, word in ((cache.desc, None), (none, cache.status), (none, None)):
        cache.refused.zero_()
        cache.status.zero_()
        assert call(ctypes.byref(cache.shape), ctypes.byref(desc), 70, x.data_ptr(), st, x.data_ptr(), st,
                    bad.data_ptr(), None, None if word is None else word.data_ptr(),
                    torch.cuda.current_stream().cuda_stream) == csa.CSA_OK
        assert csa.csa_check(cache.status) == (0 if word is None else 1)
        assert csa.csa_check(cache.refused) == (1 if desc is cache.desc else 0)
