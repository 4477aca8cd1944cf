"""Host side of the 8-bit cache: refusals (before any launch), the layout and
arithmetic of its codes, the choice of blocks (no GPU work)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import certified_sparse_attention_gb300 as csa
from oracle import kv8
from tests.gpu_common import ensure_built
from tests.test_kv4_host import I64, FAKE, Fake, HostFake, Reached, _made, no_launch, shape, status, strides  # noqa: F401

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
ODD = csa.csa_strides(4 * 8 * 128, 8 * 128, 132)    # heads at 264 bytes
FULL = csa.csa_kv8(*[FAKE] * 6)


@pytest.fixture(scope="module")
def lib():
    return ensure_built()


def cache(**kw):
    f = dict(K8=FAKE, V8=FAKE, scale=FAKE, span=FAKE, Kt=FAKE, Vt=FAKE)
    f.update(kw)
    return csa.csa_kv8(**f)


@pytest.mark.parametrize("over,want", [
    (dict(T=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(lens_dev=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=ODD), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(cache=cache(V8=None)), INVALID), (dict(cache=cache(Kt=None)), INVALID),
    (dict(cache=cache(scale=FAKE + 8)), INVALID),
    (dict(cache=cache(span=FAKE + 4)), INVALID),
    (dict(cache=cache(refused=FAKE + 2)), INVALID),
    (dict(shape=shape(n_max=0)), INVALID),
    (dict(shape=shape(d=32)), UNSUPPORTED)])
def test_append_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), T=4, k=FAKE, ks=strides(heads=2),
             v=FAKE, vs=strides(heads=2), lens_dev=FAKE, n_new=None,
             status=None, stream=0)
    a.update(over)
    assert csa.csa_kv8_append(**a) == want


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), INVALID), (dict(rows=(1 << 31) + 1), INVALID),
    (dict(lens_dev=None), INVALID), (dict(K=None), INVALID),
    (dict(V=FAKE + 8), INVALID), (dict(cache=cache(K8=None)), INVALID),
    (dict(shape=shape(Hq=32, Hkv=2)), UNSUPPORTED)])
def test_unpack_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), rows=10, first=None, lens_dev=FAKE,
             K=FAKE, V=FAKE, status=None, stream=0)
    a.update(over)
    assert csa.csa_kv8_unpack(**a) == want


DECODE = [
    (dict(T=0), INVALID), (dict(T=17), UNSUPPORTED),
    (dict(shape=shape(Hq=16), T=9), UNSUPPORTED),      # 72 rows
    (dict(q=None), INVALID), (dict(lens_dev=None), INVALID),
    (dict(o=None), INVALID), (dict(o=FAKE + 4), INVALID), (dict(qs=ODD), INVALID),
    (dict(qs=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(cache=cache(K8=FAKE + 8)), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=FAKE + 16), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE),
    (dict(shape=shape(n_max=100000), workspace_bytes=256), WORKSPACE),
    (dict(shape=shape(d=96)), UNSUPPORTED)]


@pytest.mark.parametrize("over,want", DECODE)
def test_decode_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), T=4, q=FAKE, qs=strides(),
             lens_dev=FAKE, n_q=None, o=FAKE, lse=None, workspace=FAKE,
             workspace_bytes=1 << 40, stream=0)
    a.update(over)
    assert csa.csa_kv8_decode(**a) == want


@pytest.mark.parametrize("over,want", DECODE + [
    (dict(blocks=None), INVALID), (dict(count=None), INVALID),
    (dict(blocks=FAKE + 2), INVALID), (dict(count=FAKE + 1), INVALID),
    (dict(n_sel=0), INVALID), (dict(n_sel=-1), INVALID), (dict(n_sel=1025), UNSUPPORTED)])
def test_decode_blocks_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), T=4, q=FAKE, qs=strides(),
             lens_dev=FAKE, n_q=None, blocks=FAKE, count=FAKE, n_sel=1000, o=FAKE,
             lse=None, workspace=FAKE, workspace_bytes=1 << 40, stream=0)
    a.update(over)
    assert csa.csa_kv8_decode_blocks(**a) == want


@pytest.mark.parametrize("over,want", [
    (dict(T=0), INVALID), (dict(T=17), UNSUPPORTED),
    (dict(shape=shape(Hq=16), T=9), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(lens_dev=None), INVALID), (dict(blocks=None), INVALID),
    (dict(count=None), INVALID), (dict(count=FAKE + 2), INVALID),
    (dict(qs=ODD), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(cache=cache(span=None)), INVALID), (dict(n_sel=0), INVALID),
    (dict(n_first=-1), INVALID), (dict(n_last=0), INVALID),
    (dict(n_first=7, n_last=2), INVALID), (dict(n_first=(1 << 31) - 1), INVALID),
    (dict(n_last=(1 << 31) - 1), INVALID), (dict(n_sel=1025), UNSUPPORTED),
    (dict(shape=shape(n_max=(3 << 20) + 1)), UNSUPPORTED),
    (dict(shape=shape(d=96)), UNSUPPORTED)])
def test_select_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), T=4, q=FAKE, qs=strides(),
             lens_dev=FAKE, n_q=None, n_sel=8, n_first=1, n_last=2, blocks=FAKE,
             count=FAKE, status=None, stream=0)
    a.update(over)
    assert csa.csa_kv8_select(**a) == want


def test_workspace_size(lib):
    # one word and, where an item may be cut, the parts' sums
    assert csa.csa_kv8_workspace_size(shape(n_max=500), 1) == 256
    s = shape(n_max=100000)
    assert csa.csa_kv8_workspace_size(s, 1) > 256
    assert csa.csa_kv8_workspace_size(s, 16) > csa.csa_kv8_workspace_size(s, 1)
    assert csa.csa_kv8_workspace_size(s, 1, 4) == 256
    assert csa.csa_kv8_workspace_size(s, 1, 1024) > 256
    for T, n in ((0, 0), (17, 0), (1, -1), (1, 1025)):
        assert csa.csa_kv8_workspace_size(s, T, n) == 0
    assert csa.csa_kv8_workspace_size(shape(d=96), 1) == 0
    assert csa.csa_kv8_workspace_size(shape(Hq=16), 9) == 0


@pytest.mark.parametrize("BH", [(1, 1), (2, 1), (4, 4), (2, 8), (3, 3), (19, 1), (8, 5), (16, 8)])
@pytest.mark.parametrize("G,d", [(1, 64), (2, 128), (4, 128), (8, 64)])
def test_workspace_is_enough_for_fewer_tokens_and_shorter_lists(lib, BH, G, d):
    # what was sized for T tokens and lists of n_sel blocks also serves a call of
    # fewer: more tokens are more items, which share CTAs where fewer are cut
    s = csa.make_shape(BH[0], BH[1] * G, BH[1], d, 64 * 700, "bf16")
    tokens = [t for t in range(1, 17) if t * G <= 64]
    by_lists = {}
    for n in [0] + list(range(1, 45)) + [60, 61, 80, 81, 120, 121, 160, 161, 240, 241, 320, 321, 480, 640, 1024]:
        sizes = [csa.csa_kv8_workspace_size(s, t, n) for t in tokens]
        assert min(sizes) >= 256 and sizes == sorted(sizes), n
        if n:
            by_lists[n] = sizes
    for i in range(len(tokens)):
        assert [x[i] for x in by_lists.values()] == sorted(x[i] for x in by_lists.values())


# ------------------------------------------------------------- the binding

def kv8_cache(s=None, device=0):
    import torch
    return _made(csa.KV8Cache, shape=s or shape(), device=device, status=status(), desc=FULL, dtype=torch.bfloat16)


@pytest.mark.parametrize("over", [
    dict(k=Fake([2, 4, 2, 64])), dict(v=Fake([2, 3, 2, 128])),
    dict(k=Fake([2, 4, 2, 128], "float32")), dict(lens_dev=Fake([3], I64)),
    dict(n_new=Fake([2], "int32")), dict(v=HostFake([2, 4, 2, 128])),
    dict(k=Fake([2, 4, 2, 128], stride=[1024, 256, 132, 1]))])
def test_binding_refuses_append_arguments(no_launch, over):
    a = dict(k=Fake([2, 4, 2, 128]), v=Fake([2, 4, 2, 128]), lens_dev=Fake([2], I64), n_new=None)
    with pytest.raises(Reached):
        kv8_cache().append(**a, stream=0)
    a.update(over)
    with pytest.raises(ValueError):
        kv8_cache().append(**a, stream=0)


@pytest.mark.parametrize("over", [
    dict(K=Fake([2, 2, 0, 128]), V=Fake([2, 2, 0, 128])),
    dict(V=Fake([2, 2, 6, 128])), dict(first=Fake([2], "int32"))])
def test_binding_refuses_unpack_arguments(no_launch, over):
    a = dict(K=Fake([2, 2, 5, 128]), V=Fake([2, 2, 5, 128]), lens_dev=Fake([2], I64), first=None)
    with pytest.raises(Reached):
        kv8_cache().unpack(**a, stream=0)
    a.update(over)
    with pytest.raises(ValueError):
        kv8_cache().unpack(**a, stream=0)


def operator(cls):
    import torch
    more = {} if cls is csa.KV8Decode else dict(
        n_sel=6, n_first=1, n_last=2, status=status(), blocks=Fake([2, 4, 2, 6], "int32"), count=Fake([2, 4, 2], "int32"))
    return _made(cls, shape=shape(), T=4, device=0, lse=None, o=Fake([1], "float32"), ws=Fake([1], "uint8"), ws_bytes=0,
                 dtype=torch.bfloat16, **more)


def calls(op):
    return [op] if isinstance(op, csa.KV8Decode) else [op, op.select, op.attend]


@pytest.mark.parametrize("cls", [csa.KV8Decode, csa.KV8Sparse])
@pytest.mark.parametrize("over", [
    dict(q=Fake([2, 2, 8, 128])), dict(q=Fake([2, 4, 2, 128])),
    dict(n_q=Fake([2], "int32")), dict(lens_dev=HostFake([2], I64)),
    dict(cache=kv8_cache(shape(n_max=1001))), dict(cache=kv8_cache(device=1)),
    dict(cache=_made(csa.KV4Cache, shape=shape(), desc=None, device=0))])
def test_binding_refuses_decode_arguments(no_launch, cls, over):
    for call in calls(operator(cls)):
        a = dict(q=Fake([2, 4, 8, 128]), lens_dev=Fake([2], I64), n_q=None, cache=kv8_cache())
        with pytest.raises(Reached):
            call(**a, stream=0)
        a.update(over)
        with pytest.raises(ValueError):
            call(**a, stream=0)


@pytest.mark.parametrize("blocks,count", [
    (Fake([2, 4, 2, 6], "int32"), None), (None, Fake([2, 4, 2], "int32")),
    (Fake([2, 4, 2, 6], I64), Fake([2, 4, 2], "int32")),
    (Fake([2, 4, 2, 5], "int32"), Fake([2, 4, 2], "int32")),
    (Fake([2, 4, 2, 6], "int32"), Fake([2, 4, 1], "int32")),
    (HostFake([2, 4, 2, 6], "int32"), Fake([2, 4, 2], "int32"))])
def test_binding_refuses_lists(no_launch, blocks, count):
    op = operator(csa.KV8Sparse)
    a = dict(q=Fake([2, 4, 8, 128]), lens_dev=Fake([2], I64), n_q=None, cache=kv8_cache(), stream=0)
    with pytest.raises(Reached):
        op.attend(blocks=Fake([2, 4, 2, 6], "int32"), count=Fake([2, 4, 2], "int32"), **a)
    with pytest.raises(ValueError):
        op.attend(blocks=blocks, count=count, **a)


@pytest.mark.parametrize("n_sel,first,last", [(4, -1, 2), (4, 1, 0), (4, 3, 2), (0, 0, 1)])
def test_sparse_refuses_its_parameters(n_sel, first, last):
    with pytest.raises(ValueError):
        csa.KV8Sparse(shape(), "cpu", n_sel, n_first=first, n_last=last)


@pytest.mark.parametrize("T,n_sel", [(17, 8), (1, 1025)])
def test_sparse_refuses_sizes(lib, T, n_sel):
    with pytest.raises(csa.CsaError):
        csa.KV8Sparse(shape(), "cpu", n_sel, T=T)


# -------------------------------------------------------------- the oracle

@pytest.mark.parametrize("d", [64, 128])
def test_places_are_a_permutation(d):
    assert sorted(kv8.key_places(d).ravel()) == list(range(64 * d))
    x = np.random.default_rng(0).normal(size=(64, d)).astype(np.float32)
    k8, v8, scale, span = kv8.block(x, x)
    for t in (0, 1, 17, 40, 63):
        for c in (0, 5, d - 1):
            assert k8[kv8.key_place(t, c, d)] == v8[c, t]
            assert span[1, c] <= v8[c, t] <= span[0, c]


def test_codes_stand_near_the_rows():
    # half a step, and the roundings of the quotient (127 2^-24 steps, two of
    # them) and of the product
    x = np.random.default_rng(5).normal(size=(64, 64)).astype(np.float32)
    step = kv8.steps(x)
    c = kv8.codes(x, step)
    assert np.abs(c).max() == 127 and step == np.abs(x).max() / np.float32(127)
    assert np.all(np.abs(kv8.stands_for(c, step) - x) <= step * (0.5 + 256 * 2.0 ** -24) + np.abs(x) * 2.0 ** -23)
    assert kv8.steps(0 * x) == 1 and np.all(kv8.codes(0 * x, np.float32(1)) == 0)


def test_scores_bound_what_a_block_holds():
    # with the query's own 8-bit codes, no key of a block scores above it
    rng = np.random.default_rng(6)
    d = 64
    K = rng.normal(size=(5, 64, d)).astype(np.float32)
    q = rng.normal(size=(3, d)).astype(np.float32)
    blocks = [kv8.block(x, x) for x in K]
    got = kv8.scores(q, np.stack([b[3] for b in blocks]), np.array([b[2][0] for b in blocks]))
    for j, x in enumerate(K):
        sk = kv8.steps(x)
        top = max((kv8.codes(x, sk) @ kv8.codes(h, kv8.steps(h[None]))).max() * float(sk) * float(kv8.steps(h[None])) for h in q)
        assert top <= got[j] * (1 + 2.0 ** -22)


def test_choice():
    s = np.array([5, 1, 9, 9, 2, 9, 0, 0], np.float32)
    assert kv8.choose(s, 7, 8, 1, 1) == list(range(8))
    assert kv8.choose(s, 7, 4, 1, 1) == [0, 2, 3, 7]
    assert kv8.choose(s, 7, 3, 0, 1) == [2, 3, 7]
    assert kv8.choose(s, 7, 5, 0, 4) == [2, 4, 5, 6, 7]
    assert kv8.choose(s[:3], 2, 2, 0, 1) == [0, 2]


def test_structure_matches_the_header(lib, tmp_path):
    # sizes and offsets as a C compiler has them
    cc = shutil.which("cc") or shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f for f, _ in csa.csa_kv8._fields_]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "csa.h"', "int main(void) {",
             '  printf("%zu\\n", sizeof(csa_kv8));']
    lines += [f'  printf("%zu\\n", offsetof(csa_kv8, {f}));' for f in fields]
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(csa.csa_kv8)] + [getattr(csa.csa_kv8, f).offset for f in fields]
