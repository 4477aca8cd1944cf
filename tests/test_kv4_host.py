"""Host side of csa_qk_norm_rope and the 4-bit cache: refusals (before any
launch), the rotation table, the layout of the value codes (no GPU work)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import certified_sparse_attention_gb300 as csa
from oracle import kv4
from oracle.quantize import quantize_keys
from tests.gpu_common import ensure_built

FAKE = 256          # an aligned address nothing is read from
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    return ensure_built()


def shape(**kw):
    a = dict(B=2, Hq=8, Hkv=2, d=128, n_max=1000, dtype="bf16")
    a.update(kw)
    return csa.make_shape(**a)


def strides(T=4, heads=8, d=128):
    return csa.csa_strides(T * heads * d, heads * d, d)


def cache(**kw):
    f = dict(K4=FAKE, bounds=FAKE, V4=FAKE, vscale=FAKE, Kt=FAKE, Vt=FAKE)
    f.update(kw)
    return csa.csa_kv4(**f)


def norm(**kw):
    f = dict(wq=FAKE, wk=FAKE, norm_eps=1e-6, rot_dim=128, interleaved=0,
             turns=FAKE)
    f.update(kw)
    return csa.csa_norm_rope(**f)


ODD = csa.csa_strides(4 * 8 * 128, 8 * 128, 132)    # heads at 264 bytes


@pytest.mark.parametrize("over,want", [
    (dict(T=0), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(lens_dev=None), INVALID), (dict(q_out=None), INVALID),
    (dict(K=None), INVALID), (dict(V=None), INVALID),
    (dict(qs=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(qs=ODD), INVALID),
    (dict(ks=ODD), INVALID), (dict(vs=ODD), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(q_out=FAKE + 2), INVALID),
    (dict(K=FAKE + 8), INVALID), (dict(to_cache=2), INVALID),
    (dict(params=norm(rot_dim=4)), INVALID),
    (dict(params=norm(rot_dim=136)), INVALID),
    (dict(params=norm(rot_dim=-8)), INVALID),
    (dict(params=norm(turns=None)), INVALID),
    (dict(params=norm(interleaved=2)), INVALID),
    (dict(params=norm(norm_eps=-1.0)), INVALID),
    (dict(params=norm(norm_eps=math.nan)), INVALID),
    (dict(params=norm(wq=FAKE + 4)), INVALID),
    (dict(shape=shape(d=96)), UNSUPPORTED),
    (dict(shape=shape(B=129)), UNSUPPORTED),
    (dict(shape=shape(Hq=6)), UNSUPPORTED),
    (dict(shape=shape(n_max=0)), INVALID)])
def test_norm_rope_refusals(lib, over, want):
    a = dict(shape=shape(), T=4, params=norm(), q=FAKE, qs=strides(), k=FAKE,
             ks=strides(heads=2), v=FAKE, vs=strides(heads=2), lens_dev=FAKE,
             n_new=None, q_out=FAKE, K=FAKE, V=FAKE, to_cache=1, status=None,
             stream=0)
    a.update(over)
    assert csa.csa_qk_norm_rope(**a) == want


@pytest.mark.parametrize("over,want", [
    (dict(T=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(lens_dev=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=ODD), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(cache=cache(V4=None)), INVALID),
    (dict(cache=cache(Kt=None)), INVALID),
    (dict(cache=cache(vscale=FAKE + 8)), INVALID),
    (dict(shape=shape(d=32)), UNSUPPORTED)])
def test_append_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), T=4, k=FAKE, ks=strides(heads=2),
             v=FAKE, vs=strides(heads=2), lens_dev=FAKE, n_new=None,
             status=None, stream=0)
    a.update(over)
    assert csa.csa_kv4_append(**a) == want


@pytest.mark.parametrize("over,want", [
    (dict(rows=0), INVALID), (dict(rows=(1 << 31) + 1), INVALID),
    (dict(lens_dev=None), INVALID), (dict(K=None), INVALID),
    (dict(V=FAKE + 8), INVALID), (dict(cache=cache(bounds=None)), INVALID),
    (dict(shape=shape(Hq=32, Hkv=2)), UNSUPPORTED)])
def test_unpack_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), rows=10, first=None, lens_dev=FAKE,
             K=FAKE, V=FAKE, status=None, stream=0)
    a.update(over)
    assert csa.csa_kv4_unpack(**a) == want


@pytest.mark.parametrize("over,want", [
    (dict(T=0), INVALID), (dict(T=17), UNSUPPORTED),
    (dict(shape=shape(Hq=16), T=9), UNSUPPORTED),      # 72 rows
    (dict(q=None), INVALID), (dict(lens_dev=None), INVALID),
    (dict(o=None), INVALID), (dict(qs=ODD), INVALID), (dict(qs=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(cache=cache(K4=FAKE + 8)), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace=FAKE + 16), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE),
    (dict(shape=shape(n_max=100000), workspace_bytes=256), WORKSPACE),
    (dict(shape=shape(d=96)), UNSUPPORTED)])
def test_decode_refusals(lib, over, want):
    a = dict(shape=shape(), cache=cache(), T=4, q=FAKE, qs=strides(),
             lens_dev=FAKE, n_q=None, o=FAKE, lse=None, workspace=FAKE,
             workspace_bytes=1 << 40, stream=0)
    a.update(over)
    assert csa.csa_kv4_decode(**a) == want


def test_workspace_size(lib):
    # one word and, where a sequence may be cut, the parts' sums
    assert csa.csa_kv4_workspace_size(shape(), 1) == 256
    s = shape(n_max=100000)
    assert csa.csa_kv4_workspace_size(s, 1) > 256
    assert csa.csa_kv4_workspace_size(s, 16) > csa.csa_kv4_workspace_size(s, 1)
    assert csa.csa_kv4_workspace_size(s, 0) == 0
    assert csa.csa_kv4_workspace_size(s, 17) == 0
    assert csa.csa_kv4_workspace_size(shape(d=96), 1) == 0
    assert csa.csa_kv4_workspace_size(shape(Hq=16), 9) == 0


def test_rope_turns_are_exact(lib):
    # within one unit of 2^-64 turn of inv_freq / (2 pi), modulo one turn
    rng = np.random.default_rng(3)
    f = np.concatenate([500000.0 ** (-np.arange(64) / 64), [0.0, -0.25, 7.0,
                        -1e-9, 2.0 ** 20], rng.normal(size=50)])
    got = csa.csa_rope_turns(f)
    for x, u in zip(f, got):
        want = Fraction(float(x)) / (2 * kv4.PI) * 2 ** 64
        off = (want - u) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, x
    for bad in ([math.nan], [math.inf], [2.0 ** 21]):
        with pytest.raises(csa.CsaError):
            csa.csa_rope_turns(bad)


def test_struct_layouts_match_the_header(lib, tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("cc") or shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = (csa.csa_strides, csa.csa_norm_rope, csa.csa_kv4)
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "csa.h"',
             "int main(void) {"]
    for st in structs:
        nm = st.__name__
        lines.append(f'  printf("%zu\\n", sizeof({nm}));')
        for f, _ in st._fields_:
            lines.append(f'  printf("%zu\\n", offsetof({nm}, {f}));')
    lines += ["  return 0;", "}"]
    (tmp_path / "l.c").write_text("\n".join(lines) + "\n")
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I",
                    os.path.join(root, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run(
        [str(tmp_path / "l")], capture_output=True, text=True,
        check=True).stdout.split()]
    want = []
    for st in structs:
        want.append(ctypes.sizeof(st))
        want += [getattr(st, f).offset for f, _ in st._fields_]
    assert got == want


class Fake:
    """Stands in for a CUDA tensor in host-only checks."""

    def __init__(self, size, dtype="bfloat16", stride=None, device=0,
                 at=FAKE):
        import torch
        self.shape, self.dtype = torch.Size(size), getattr(torch, dtype)
        self.dev, self.at = device, at
        st, n = [], 1
        for x in reversed(size):
            st.insert(0, n)
            n *= x
        self.st = tuple(stride or st)
        self.contig = stride is None

    def get_device(self):
        return self.dev

    def stride(self):
        return self.st

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self.contig

    def data_ptr(self):
        return self.at


def HostFake(*a, **k):
    return Fake(*a, device=-1, **k)


def _made(cls, **kw):
    """An object as its constructor leaves it, without device memory."""
    x = cls.__new__(cls)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


I64 = "int64"


class Reached(Exception):
    pass


@pytest.fixture
def no_launch(monkeypatch):
    """A call that would reach the library raises; device 0 is current."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class Library:
        def __getattr__(self, name):
            def call(*a):
                raise Reached(name)
            return call
    monkeypatch.setattr(csa, "load_library", lambda: Library())


def status():
    return Fake([4], "int32")


@pytest.mark.parametrize("over", [
    dict(q=Fake([2, 4, 8, 64])), dict(q=Fake([2, 8, 128])),
    dict(q=Fake([2, 4, 8, 128], "float16")),
    dict(q=Fake([2, 4, 8, 128], device=1)),
    dict(q=HostFake([2, 4, 8, 128])),
    dict(q=Fake([2, 4, 8, 128], at=FAKE + 2)),
    dict(q=Fake([2, 4, 8, 128], stride=[4096, 1024, 1, 8])),
    dict(q=Fake([2, 4, 8, 128], stride=[4096, 1024, 132, 1])),
    dict(k=Fake([2, 3, 2, 128])), dict(v=Fake([2, 4, 8, 128])),
    dict(v=None), dict(V=None), dict(K=Fake([2, 2, 999, 128])),
    dict(K=Fake([2, 2, 1000, 128], "float32")),
    dict(lens_dev=Fake([2], "int32")), dict(lens_dev=Fake([3], I64)),
    dict(lens_dev=HostFake([2], I64)), dict(n_new=Fake([1], I64)),
    dict(lens_dev=Fake([2], "uint64")), dict(n_new=Fake([2], "float64")),
    dict(q_out=None), dict(q_out=Fake([2, 4, 2, 128])),
    dict(q_out=Fake([2, 4, 8, 128], stride=[8192, 2048, 256, 1]))])
def test_binding_refuses_rope_arguments(no_launch, over):
    import torch
    op = _made(csa.QKNormRope, shape=shape(), device=0, status=status(),
               params=norm(), dtype=torch.bfloat16)
    a = dict(q=Fake([2, 4, 8, 128]), k=Fake([2, 4, 2, 128]),
             v=Fake([2, 4, 2, 128]), K=Fake([2, 2, 1000, 128]),
             V=Fake([2, 2, 1000, 128]), lens_dev=Fake([2], I64),
             n_new=Fake([2], I64), q_out=Fake([2, 4, 8, 128]))
    with pytest.raises(Reached):
        op(**a, stream=0)
    a.update(over)
    with pytest.raises(ValueError):
        op(**a, stream=0)


@pytest.mark.parametrize("over", [
    dict(k=Fake([2, 4, 3, 128])), dict(v=Fake([2, 5, 2, 128])),
    dict(k=Fake([2, 0, 2, 128])), dict(v=HostFake([2, 4, 2, 128])),
    dict(lens_dev=Fake([2], I64, device=1)),
    dict(n_new=Fake([2], "float32"))])
def test_binding_refuses_append_arguments(no_launch, over):
    import torch
    op = _made(csa.KV4Cache, shape=shape(), device=0, status=status(),
               desc=cache(), dtype=torch.bfloat16)
    a = dict(k=Fake([2, 4, 2, 128]), v=Fake([2, 4, 2, 128]),
             lens_dev=Fake([2], I64), n_new=None)
    with pytest.raises(Reached):
        op.append(**a, stream=0)
    a.update(over)
    with pytest.raises(ValueError):
        op.append(**a, stream=0)


@pytest.mark.parametrize("over", [
    dict(K=Fake([2, 2, 0, 128]), V=Fake([2, 2, 0, 128])),
    dict(V=Fake([2, 2, 6, 128])), dict(K=Fake([2, 2, 5, 64])),
    dict(K=Fake([2, 2, 5, 128], stride=[9999, 640, 128, 1])),
    dict(V=Fake([2, 2, 5, 128], "float32")),
    dict(first=Fake([2], "int32"))])
def test_binding_refuses_unpack_arguments(no_launch, over):
    import torch
    op = _made(csa.KV4Cache, shape=shape(), device=0, status=status(),
               desc=cache(), dtype=torch.bfloat16)
    a = dict(K=Fake([2, 2, 5, 128]), V=Fake([2, 2, 5, 128]),
             lens_dev=Fake([2], I64), first=None)
    with pytest.raises(Reached):
        op.unpack(**a, stream=0)
    a.update(over)
    with pytest.raises(ValueError):
        op.unpack(**a, stream=0)


@pytest.mark.parametrize("over", [
    dict(q=Fake([2, 2, 8, 128])), dict(q=Fake([2, 4, 2, 128])),
    dict(n_q=Fake([2], "int32")), dict(lens_dev=HostFake([2], I64)),
    dict(cache=_made(csa.KV4Cache, shape=shape(n_max=1001), desc=cache(),
                     device=0)),
    dict(cache=_made(csa.KV4Cache, shape=shape(), desc=cache(),
                     device=1))])
def test_binding_refuses_decode_arguments(no_launch, over):
    import torch
    op = _made(csa.KV4Decode, shape=shape(), T=4, device=0, lse=None,
               o=Fake([1], "float32"), ws=Fake([1], "uint8"), ws_bytes=0,
               dtype=torch.bfloat16)
    a = dict(q=Fake([2, 4, 8, 128]), lens_dev=Fake([2], I64), n_q=None,
             cache=_made(csa.KV4Cache, shape=shape(), desc=cache(), device=0))
    with pytest.raises(Reached):
        op(**a, stream=0)
    a.update(over)
    with pytest.raises(ValueError):
        op(**a, stream=0)


def test_another_current_device_is_refused(no_launch, monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    op = _made(csa.KV4Cache, shape=shape(), device=0, status=status(),
               desc=cache(), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        op.append(Fake([2, 4, 2, 128]), Fake([2, 4, 2, 128]),
                  Fake([2], I64), stream=0)


def test_value_places_are_a_permutation():
    assert sorted(kv4.v4_place(t) for t in range(64)) == list(range(64))
    codes = np.random.default_rng(0).integers(0, 16, (64, 8)).astype(np.uint8)
    packed = kv4.pack_values(codes)
    for t in range(64):
        p = kv4.v4_place(t)
        assert np.array_equal((packed[:, p // 2] >> (4 * (p & 1))) & 15,
                              codes[t])


def test_codes_stand_near_the_rows():
    # |v - stands_for| <= Delta / 2 and float32 rounding, keys and values;
    # constant rows are exact
    rng = np.random.default_rng(5)
    x = rng.normal(size=(64, 32)).astype(np.float32)
    x[3] = 1.25
    c, m, dl = kv4.quantize_values(x)
    got = kv4.stands_for(c, m[:, None], dl[:, None])
    # half a step, plus the roundings of the quotient (15 * 2^-24 steps, four
    # of them) and of the sum
    lim = dl[:, None] * (0.5 + 60 * 2.0 ** -24) + np.abs(x).max() * 2.0 ** -22
    assert np.all(np.abs(got - x) <= lim)
    assert np.all(got[3] == x[3]) and dl[3] == 0 and c.max() == 15
    codes, _, m, dl = quantize_keys(x, 64)
    got = kv4.stands_for(codes, m[0], dl[0])
    lim = dl[0] * (0.5 + 60 * 2.0 ** -24) + np.abs(x).max() * 2.0 ** -22
    assert np.all(np.abs(got - x) <= lim)


def test_rotation_keeps_norms_and_relative_angles():
    # a rotated q . k depends on the distance alone
    rng = np.random.default_rng(6)
    f = 10000.0 ** (-np.arange(16) / 16)
    q, k = rng.normal(size=(2, 32))
    for inter in (False, True):
        base = kv4.norm_rope(q, None, 0, 5, f, inter) @ \
            kv4.norm_rope(k, None, 0, 2, f, inter)
        far = kv4.norm_rope(q, None, 0, 2 ** 31 + 5, f, inter) @ \
            kv4.norm_rope(k, None, 0, 2 ** 31 + 2, f, inter)
        assert abs(base - far) < 1e-12
        assert abs(np.linalg.norm(kv4.norm_rope(q, None, 0, 77, f, inter)) -
                   np.linalg.norm(q)) < 1e-12
    ones = kv4.norm_rope(q, np.ones(32), 0.0, 0, [], False)
    assert abs(np.mean(ones ** 2) - 1) < 1e-12


def test_word_of_refusals_is_checked(lib):
    for bad in (FAKE + 1, FAKE + 2):
        c = cache(refused=bad)
        assert csa.csa_kv4_append(shape(), c, 4, FAKE, strides(heads=2), FAKE,
                                  strides(heads=2), FAKE, None, None,
                                  0) == INVALID
        assert csa.csa_kv4_unpack(shape(), c, 10, None, FAKE, FAKE, FAKE, None,
                                  0) == INVALID
        assert csa.csa_kv4_decode(shape(), c, 4, FAKE, strides(), FAKE, None,
                                  FAKE, None, FAKE, 1 << 40, 0) == INVALID
