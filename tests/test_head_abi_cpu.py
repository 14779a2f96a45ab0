"""The C ABI of 4-bit products, sampling and verification without a GPU:
exports, layouts, and every refusal that the host makes before it touches the
device."""

import ctypes
import os
import re
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", h) for h in ("peagle_w4.h", "peagle_sample.h")]
BASE = 1 << 20     # host addresses stand in for device pointers: a refused call reads none


@pytest.fixture(scope="module")
def B():
    from speculative_drafting_expand_gb300 import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    binding.lib()
    return binding


def test_library_exports_every_declared_symbol(B):
    text = "".join(open(h).read() for h in HEADERS)
    fns = sorted(set(re.findall(r"^(?:pe_status|int64_t)\s+(pe_\w+)\(", text, re.M)))
    assert set(fns) == set(B.HEAD_EXPORTED)
    assert all(hasattr(B.lib(), f) for f in fns)


def test_dist_layout_matches_the_header(B):
    src = r"""
    #include <stdio.h>
    #include <stddef.h>
    #include "peagle_w4.h"
    #include "peagle_sample.h"
    int main(void) {
      printf("%zu %zu %zu %zu %zu %d\n", sizeof(pe_dist), offsetof(pe_dist, cut),
             offsetof(pe_dist, cut_token), offsetof(pe_dist, total), offsetof(pe_dist, token),
             PE_DEV_BAD_TOKEN);
      return 0;
    }
    """
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    D = B.pe_dist
    assert got == [ctypes.sizeof(D), D.cut.offset, D.cut_token.offset, D.total.offset,
                   D.token.offset, B.PE_DEV_BAD_TOKEN]


SIZES = [(dict(n=0), 1), (dict(k=0), 1), (dict(group=16), 1), (dict(group=256), 1),
         (dict(n=-3), 1), (dict(k=(1 << 18) + 1), 2), (dict(n=(1 << 24) + 1), 2)]


def _call(fn, defaults, change):
    f = dict(defaults)
    assert set(change) <= set(f)
    f.update(change)
    return fn(*f.values())


def _pack(B, **change):
    return _call(B.lib().pe_w4_pack, dict(codes=BASE, scales=BASE, n=17, k=70, group=32,
                                          packed=BASE, stream=0), change)


def _quantize(B, **change):
    return _call(B.lib().pe_w4_quantize, dict(w=BASE, dtype=0, stride=70, n=17, k=70, group=32,
                                              packed=BASE, stream=0), change)


def _linear(B, **change):
    return _call(B.lib().pe_w4_linear, dict(packed=BASE, n=17, k=70, group=32, rows=3, xd=0,
                                            x=BASE, xs=70, yd=1, y=BASE, ys=17, stream=0), change)


@pytest.mark.parametrize("change,status", SIZES)
def test_w4_sizes_are_refused_by_every_call(B, change, status):
    big = dict(stride=1 << 30) if "k" in change else {}
    assert _pack(B, **change) == status
    assert _quantize(B, **change, **big) == status
    wide = dict(xs=1 << 30, ys=1 << 30)
    assert _linear(B, **change, **wide) == status
    s = dict(n=17, k=70, group=32)
    s.update(change)
    assert B.lib().pe_w4_bytes(s["n"], s["k"], s["group"]) == 0


def test_w4_longest_row(B):
    k = (1 << 17) + 1
    assert B.lib().pe_w4_bytes(17, k - 1, 32) > 0 and B.lib().pe_w4_bytes(17, k, 32) == 0
    assert _pack(B, k=k) == _quantize(B, k=k, stride=k) == _linear(B, k=k, xs=k, ys=17) == 2


def test_w4_bytes_is_16_rows_by_64_inputs_and_scales(B):
    f = B.lib().pe_w4_bytes
    assert f(1, 1, 32) == 512 + 64
    assert f(16, 64, 32) == 512 + 64
    assert f(17, 65, 64) == 2 * 2 * 512 + 2 * 2 * 32
    assert f(201088, 2880, 32) == 201088 * 2880 // 2 + 201088 * 90 * 2
    assert f(16, 65, 32) == 2 * 512 + 4 * 32 and f(16, 65, 128) == 2 * 512 + 32


@pytest.mark.parametrize("change", [dict(codes=0), dict(scales=0), dict(packed=0),
                                    dict(packed=BASE + 8), dict(scales=BASE + 1)])
def test_w4_pack_refusals(B, change):
    assert _pack(B, **change) == 1


@pytest.mark.parametrize("change", [dict(w=0), dict(w=BASE + 1), dict(dtype=1, w=BASE + 2),
                                    dict(dtype=2), dict(stride=69), dict(packed=BASE + 4)])
def test_w4_quantize_refusals(B, change):
    assert _quantize(B, **change) == 1


@pytest.mark.parametrize("change", [
    dict(rows=0), dict(xd=2), dict(yd=2), dict(xd=1, yd=0), dict(x=0), dict(y=0), dict(packed=0),
    dict(packed=BASE + 2), dict(xs=69), dict(ys=16), dict(x=BASE + 1), dict(y=BASE + 2),
    dict(xd=1, x=BASE + 2)])
def test_w4_linear_refusals(B, change):
    assert _linear(B, **change) == 1


def _sample(B, **change):
    return _call(B.lib().pe_sample, dict(rows=3, vocab=100, dtype=1, logits=BASE, stride=100,
                                         t=0, k=0, p=0, mp=0, u=BASE, tokens=BASE, lp=0, dist=0,
                                         stream=0), change)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), 1), (dict(vocab=0), 1), (dict(dtype=2), 1), (dict(logits=0), 1),
    (dict(logits=BASE + 2), 1), (dict(stride=99), 1), (dict(u=0), 1), (dict(tokens=0), 1),
    (dict(dist=BASE + 8), 1), (dict(vocab=393217, stride=393217), 2)])
def test_sample_refusals(B, change, status):
    assert _sample(B, **change) == status


def _verify(binding, **change):
    return _call(binding.lib().pe_verify, dict(
        B=2, T=5, vocab=100, dtype=1, logits=BASE, stride=100, ids=BASE, cu=BASE, t=0, k=0, p=0,
        mp=0, au=BASE, u=BASE, dl=0, ds=0, dd=0, acc=BASE, ids_out=BASE, lp=0, dist=BASE, err=0,
        stream=0), change)


@pytest.mark.parametrize("change,status", [
    (dict(B=0), 1), (dict(T=1), 1), (dict(vocab=0), 1), (dict(dtype=3), 1), (dict(logits=0), 1),
    (dict(stride=64), 1), (dict(ids=0), 1), (dict(cu=0), 1), (dict(au=0), 1), (dict(u=0), 1),
    (dict(acc=0), 1), (dict(ids_out=0), 1), (dict(dist=0), 1), (dict(dist=BASE + 4), 1),
    (dict(dl=BASE, ds=100), 1), (dict(dl=BASE, ds=99, dd=BASE), 1),
    (dict(dl=BASE + 2, ds=100, dd=BASE), 1), (dict(dl=BASE, ds=100, dd=BASE + 8), 1),
    (dict(vocab=1 << 19, stride=1 << 19), 2)])
def test_verify_refusals(B, change, status):
    assert _verify(B, **change) == status


def test_python_refusals(B):
    import torch
    codes = torch.zeros(16, 32, dtype=torch.uint8)
    scales = torch.zeros(16, 2, dtype=torch.bfloat16)
    for bad in ((codes.int(), scales, 64, 32), (codes[:, :31], scales, 64, 32),
                (codes, scales.float(), 64, 32), (codes, scales[:8], 64, 32),
                (codes, scales, 64, 48), (codes, scales, 0, 32), (codes.t(), scales, 64, 32),
                (codes, scales, 1 << 33, 32)):
        with pytest.raises(ValueError):
            B.W4Weight(*bad)
    with pytest.raises(ValueError, match="GPU"):
        B.W4Weight(codes, scales, 64, 32)
    with pytest.raises(ValueError, match="GPU"):
        B.W4Weight.quantize(torch.zeros(4, 64))
    for bad in (torch.zeros(4), torch.zeros(4, 64, dtype=torch.float16), torch.zeros(64, 4).t()):
        with pytest.raises(ValueError):
            B.W4Weight.quantize(bad)
    x, u = torch.zeros(3, 50), torch.zeros(3)
    for kw in (dict(logits=x.half()), dict(logits=x[0]), dict(logits=torch.zeros(50, 3).t()),
               dict(u=u[:2]), dict(u=u.double()), dict(temperature=u[:1]), dict(top_k=u),
               dict(top_p=u.double()), dict(min_p=torch.zeros(6)[::2]),
               dict(tokens=torch.zeros(3)), dict(dist=torch.zeros(3, 8))):
        a = dict(logits=x, u=u)
        a.update(kw)
        with pytest.raises(ValueError):
            B.pe_sample(**a)
    with pytest.raises(ValueError, match="GPU"):
        B.pe_sample(x, u)
    i32 = torch.int32
    ok = dict(logits=torch.zeros(5, 50), ids=torch.zeros(5, dtype=i32),
              cu_in=torch.zeros(3, dtype=i32), accept_u=torch.zeros(5), u=torch.zeros(2))
    for kw in (dict(ids=torch.zeros(4, dtype=i32)), dict(cu_in=torch.zeros(3)),
               dict(accept_u=torch.zeros(2)), dict(u=torch.zeros(5)),
               dict(temperature=torch.ones(5)), dict(draft_logits=torch.zeros(3, 50)),
               dict(draft_dist=torch.zeros(3, 8, dtype=i32)),
               dict(draft_logits=torch.zeros(3, 50).bfloat16(),
                    draft_dist=torch.zeros(3, 8, dtype=i32)),
               dict(draft_logits=torch.zeros(2, 50), draft_dist=torch.zeros(3, 8, dtype=i32)),
               dict(err=torch.zeros(2, dtype=i32))):
        with pytest.raises(ValueError):
            B.pe_verify(**dict(ok, **kw))
    with pytest.raises(ValueError, match="GPU"):
        B.pe_verify(**ok)
