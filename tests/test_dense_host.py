"""CPU tests of the dense operators' refusals: every argument error comes back before anything
is enqueued, so no device is needed (the addresses are never dereferenced)."""
import ctypes

import pytest

A = 1 << 30  # an aligned address
B = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from token_top_expert_b200 import build
    build.build()
    import token_top_expert_b200 as m
    return m.load_library()


@pytest.fixture(scope="module")
def st():
    from token_top_expert_b200 import _lib
    return _lib


def weights(st, **kw):
    v = dict(data=A, stride_group=64 * 128, stride_part=0, stride_n=128, stride_k=1)
    v.update(kw)
    return st.MsbGroupWeights(**v)


def matmul(lib, st, w=None, fn="msb_grouped_matmul", **kw):
    v = dict(x=B, ldx=128, x_rows=10, rows=None, offsets=A, groups=4, out_rows=10, n=64, k=128, out=2 * B,
             out_type=0, ldo=64)
    v.update(kw)
    i8, parts = "int8" in fn, "swiglu" in fn
    args = [v["x"], v["ldx"]] + ([v.get("xs", A)] if i8 else [])
    args += [v["x_rows"], v["rows"], v["offsets"], v["groups"], v["out_rows"],
             None if w == "null" else ctypes.byref(w or weights(st))]
    args += ([v.get("ws", A)] if i8 else []) + [v["n"], v["k"], v["out"]]
    args += ([] if parts else [v["out_type"]]) + [v["ldo"], None]
    return getattr(lib, fn)(*args)


BAD = [dict(x=None), dict(out=None), dict(x=B + 2), dict(groups=0), dict(out_rows=-1), dict(x_rows=-1),
       dict(n=0), dict(k=0), dict(offsets=None), dict(out_type=2), dict(ldo=63), dict(ldx=-8),
       dict(ldx=1 << 28), dict(ldo=1 << 28), dict(ldx=132), dict(out=B + 64), dict(out=A + 128),
       dict(rows=A + 2), dict(offsets=A + 1), dict(out=2 * B + 1)]


@pytest.mark.parametrize("kw", BAD, ids=str)
@pytest.mark.parametrize("fn", ["msb_grouped_matmul", "msb_int8_matmul", "msb_grouped_swiglu", "msb_int8_swiglu"])
def test_grouped_refusals(lib, st, fn, kw):
    if "out_type" in kw and "swiglu" in fn:
        pytest.skip("no out_type")
    w = weights(st, stride_part=64 * 128, stride_group=2 * 64 * 128)
    assert matmul(lib, st, w, fn, **kw) == st.MSB_EINVAL


def test_grouped_weight_refusals(lib, st):
    assert matmul(lib, st, "null") == st.MSB_EINVAL
    for kw in (dict(data=None), dict(data=A + 8), dict(stride_k=2), dict(stride_n=0), dict(stride_n=-128),
               dict(stride_n=129), dict(stride_group=0), dict(stride_group=4), dict(stride_n=1 << 40),
               dict(stride_n=1, stride_k=100), dict(stride_n=1, stride_k=-64)):
        assert matmul(lib, st, weights(st, **kw)) == st.MSB_EINVAL, kw
    # n-contiguous weights: the bf16 product only
    m = weights(st, stride_n=1, stride_k=64)
    assert matmul(lib, st, m, "msb_grouped_swiglu") == st.MSB_EINVAL
    assert matmul(lib, st, m, "msb_int8_matmul") == st.MSB_EUNSUPPORTED
    # gate and up need a part stride
    assert matmul(lib, st, weights(st), "msb_grouped_swiglu") == st.MSB_EINVAL
    for fn in ("msb_int8_matmul", "msb_int8_swiglu"):
        w = weights(st, stride_part=64 * 128, stride_group=2 * 64 * 128)
        assert matmul(lib, st, w, fn, xs=None) == st.MSB_EINVAL
        assert matmul(lib, st, w, fn, ws=None) == st.MSB_EINVAL


def test_grouped_limits_and_empty(lib, st):
    assert matmul(lib, st, groups=513) == st.MSB_EUNSUPPORTED
    assert matmul(lib, st, n=(1 << 20) + 1, ldo=1 << 21) == st.MSB_EUNSUPPORTED
    assert matmul(lib, st, k=(1 << 20) + 1) == st.MSB_EUNSUPPORTED
    assert matmul(lib, st, out_rows=(1 << 30) + 1, x_rows=(1 << 30) + 1) == st.MSB_EUNSUPPORTED
    assert matmul(lib, st, fn="msb_int8_matmul", k=st.MSB_INT8_MAX_K + 1) == st.MSB_EUNSUPPORTED
    # no rows: nothing to do, nothing launched
    assert matmul(lib, st, out_rows=0, x_rows=0, x=None, out=None) == st.MSB_OK


def test_route_refusals(lib, st):
    def call(**kw):
        v = dict(logits=A, t=0, ld=64, mask=None, tokens=100, experts=64, top_e=8, renorm=1, ids=B,
                 weights=2 * B, offsets=3 * B, rows=4 * B, pos=5 * B, ws=6 * B, nb=1 << 30)
        v.update(kw)
        return lib.msb_route(*v.values(), None)
    for kw in (dict(logits=None), dict(t=2), dict(ld=63), dict(ld=-1), dict(tokens=-1), dict(experts=0),
               dict(top_e=0), dict(top_e=65), dict(renorm=2), dict(ids=None), dict(weights=None),
               dict(offsets=None), dict(rows=None), dict(pos=None), dict(ws=None),
               dict(nb=lib.msb_route_workspace_size(100, 64) - 1), dict(logits=A + 1), dict(ids=B + 2),
               dict(pos=B + 1)):
        assert call(**kw) == st.MSB_EINVAL, kw
    for kw in (dict(tokens=(1 << 20) + 1), dict(experts=513, ld=600), dict(top_e=17)):
        assert call(**kw) == st.MSB_EUNSUPPORTED, kw
    assert lib.msb_route_workspace_size(100, 0) == 0 and lib.msb_route_workspace_size(-1, 8) == 0
    assert lib.msb_route_workspace_size((1 << 20) + 1, 8) == 0


def test_quantize_refusals(lib, st):
    def call(**kw):
        v = dict(x=A, t=0, ldx=128, rows=10, k=100, q=B, ldq=112, scale=2 * B)
        v.update(kw)
        return lib.msb_int8_quantize(*v.values(), None)
    for kw in (dict(x=None), dict(t=3), dict(ldx=-1), dict(rows=-1), dict(k=0), dict(q=None), dict(ldq=99),
               dict(scale=None), dict(q=A + 64), dict(scale=A + 64), dict(scale=B + 64), dict(x=A + 1), dict(scale=2 * B + 2)):
        assert call(**kw) == st.MSB_EINVAL, kw
    assert call(rows=0, x=None, q=None, scale=None) == st.MSB_OK


def test_int8_linear_refusals(lib, st):
    nb = lib.msb_int8_linear_workspace_size(10, 100)
    assert nb == 10 * (112 + 4)
    assert lib.msb_int8_linear_workspace_size(0, 1) == 16
    assert lib.msb_int8_linear_workspace_size(-1, 8) == lib.msb_int8_linear_workspace_size(1, 0) == 0
    assert lib.msb_int8_linear_workspace_size(1, st.MSB_INT8_MAX_K + 1) == 0

    def call(w=None, **kw):
        v = dict(x=B, xt=0, ldx=100, xr=10, rows=None, offsets=None, groups=1, r=10)
        u = dict(ws=A, n=64, k=100, swiglu=0, out=2 * B, ot=0, ldo=64, work=3 * B, nb=nb)
        for k, val in kw.items():
            (v if k in v else u)[k] = val
        w = w or weights(st, stride_n=112)
        return lib.msb_int8_linear(*v.values(), ctypes.byref(w), *u.values(), None)
    for kw in (dict(x=None), dict(xt=2), dict(ldx=-1), dict(xr=-1), dict(k=0), dict(swiglu=2), dict(work=None),
               dict(work=3 * B + 8), dict(nb=nb - 1), dict(x=B + 1), dict(work=B + 64), dict(out=B + 64),
               dict(out=3 * B + 64), dict(ws=None), dict(n=0), dict(swiglu=1, ot=1), dict(r=11)):
        assert call(**kw) == st.MSB_EINVAL, kw
    assert call(k=st.MSB_INT8_MAX_K + 1) == st.MSB_EUNSUPPORTED
    assert call(weights(st, stride_n=1, stride_k=64)) == st.MSB_EUNSUPPORTED


def test_header_is_plain_c(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "h.c"
    src.write_text('#include "msb_dense.h"\nint main(void) { msb_group_weights w = {0, 0, 0, 0, 1}; return (int)w.stride_k - 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only",
                    "-I", os.path.join(root, "include"), str(src)], check=True)


def test_combine_refusals(lib, st):
    def call(**kw):
        v = dict(y=A, t=0, ldy=128, yr=20, pos=B, w=2 * B, tokens=5, top_e=4, d=128, out=3 * B, ldo=128)
        v.update(kw)
        return lib.msb_combine(*v.values(), None)
    for kw in (dict(y=None), dict(t=-1), dict(ldy=-1), dict(yr=-1), dict(pos=None), dict(w=None),
               dict(tokens=-1), dict(top_e=0), dict(d=0), dict(out=None), dict(ldo=127), dict(out=A + 256),
               dict(pos=B + 2), dict(out=3 * B + 1)):
        assert call(**kw) == st.MSB_EINVAL, kw
    assert call(tokens=0, out=None, pos=None, w=None) == st.MSB_OK


def test_block_norm_refusals(lib, st):
    def call(**kw):
        v = dict(h=A, ht=1, ldh=128, y=2 * A, yt=0, ldy=128, pre=3 * A, post=4 * A, wt=0, pn=1, gate=5 * A,
                 gt=0, gr=0, gc=1, skip=1.0, res=1.0, eps=1e-6, ho=6 * A, ldho=128, x=7 * A, ldx=128,
                 rows=10, d=128)
        v.update(kw)
        return lib.msb_block_norm(*v.values(), None)
    for kw in (dict(h=None), dict(ht=2), dict(yt=2), dict(wt=2), dict(gt=2), dict(pn=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(rows=-1), dict(d=0), dict(ldh=-1), dict(ldho=127), dict(ldx=127),
               dict(gr=-1), dict(gc=-1), dict(ho=None, x=None), dict(y=None), dict(pn=0),
               dict(ho=A, ldho=256), dict(ho=A + 64), dict(x=A + 64), dict(x=2 * A + 64), dict(ho=2 * A),
               dict(h=A + 2), dict(y=2 * A + 1), dict(gate=5 * A + 1), dict(pre=3 * A + 1), dict(x=7 * A + 1),
               dict(x=6 * A + 64), dict(x=5 * A), dict(ho=3 * A), dict(x=4 * A)):
        assert call(**kw) == st.MSB_EINVAL, kw
    assert call(d=st.MSB_NORM_MAX_D + 1, ldho=1 << 15, ldx=1 << 15) == st.MSB_EUNSUPPORTED
    assert call(rows=0) == st.MSB_OK


def test_dense_block_refusals(lib, st):
    dims = st.MsbDims(256, 512, 8, 2, 16, 1)
    nb = lib.msb_dense_workspace_size(ctypes.byref(dims), 100, 0)
    assert nb > 0

    def call(**kw):
        v = dict(x=A, tokens=100, mask=None, router=2 * A, rec=3 * A, out=4 * A, dims=dims, ws=5 * A, nb=nb)
        v.update(kw)
        v["dims"] = v["dims"] and ctypes.byref(v["dims"])
        return lib.moe_dense_block(*v.values(), None)
    for kw in (dict(x=None), dict(router=None), dict(rec=None), dict(out=None), dict(ws=None), dict(dims=None),
               dict(tokens=-1), dict(nb=nb - 1), dict(x=A + 8), dict(rec=A + 2), dict(ws=5 * A + 8),
               dict(out=A + 512), dict(out=5 * A + 512), dict(dims=st.MsbDims(250, 512, 8, 2, 16, 1)),
               dict(dims=st.MsbDims(256, 512, 8, 9, 16, 1)), dict(dims=st.MsbDims(256, 512, 8, 2, 16, 2))):
        assert call(**kw) == st.MSB_EINVAL, kw
    assert call(tokens=(1 << 20) + 1) == st.MSB_EUNSUPPORTED
    assert call(dims=st.MsbDims(8256, 512, 8, 2, 16, 1)) == st.MSB_EUNSUPPORTED
    assert call(tokens=0) == st.MSB_OK
    i8 = lib.msb_dense_workspace_size(ctypes.byref(dims), 100, 1)
    assert i8 > nb
    args = [A, 100, None, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, ctypes.byref(dims), 8 * A, i8, None]
    for at in (3, 4, 5, 6, 7, 8, 10):
        bad = list(args)
        bad[at] = None
        assert lib.moe_dense_block_int8(*bad) == st.MSB_EINVAL, at
    assert lib.msb_dense_workspace_size(ctypes.byref(dims), -1, 0) == 0
    assert lib.msb_dense_workspace_size(None, 1, 0) == 0


def test_binding_refusals():
    """What the binding sees before the C call: types, shapes, strides, devices."""
    import torch

    import token_top_expert_b200 as msb
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w, offs = torch.zeros(6, 32, dtype=bf), torch.zeros(2, 8, 32, dtype=bf), torch.zeros(3, dtype=i32)
    cases = [
        lambda: msb.grouped_matmul(x.float(), w, offs),
        lambda: msb.grouped_matmul(x, w.float(), offs),
        lambda: msb.grouped_matmul(x[:, :16], w, offs),
        lambda: msb.grouped_matmul(x, w),                                   # offsets missing
        lambda: msb.grouped_matmul(x, w, offs.long()),
        lambda: msb.grouped_matmul(x, w, offs[:2]),
        lambda: msb.grouped_matmul(x, w, offs, rows=torch.zeros(4)),
        lambda: msb.grouped_matmul(x.t(), w, offs),
        lambda: msb.grouped_matmul(x, w, offs, out=torch.zeros(6, 7, dtype=bf)),
        lambda: msb.grouped_matmul(x, w, offs, out=torch.zeros(5, 8, dtype=bf)),
        lambda: msb.grouped_matmul(x, w, offs, out=torch.zeros(6, 8, dtype=torch.float16)),
        lambda: msb.grouped_matmul(x, w, offs, out=torch.zeros(6, 8, dtype=bf), out_dtype=f32),
        lambda: msb.grouped_matmul(x, w[None, None], offs),
        lambda: msb.grouped_matmul(x, w, offs),                             # CPU tensors
        lambda: msb.grouped_swiglu(x, w[:, None], offs),
        lambda: msb.grouped_swiglu(x, torch.zeros(2, 2, 8, 32, dtype=bf), offs, out=torch.zeros(6, 8)),
        lambda: msb.matmul_int8(x.char(), torch.zeros(5), w.char(), torch.zeros(2, 8), offs),
        lambda: msb.matmul_int8(x.char(), torch.zeros(6), w.char(), torch.zeros(2, 7), offs),
        lambda: msb.quantize_int8(x, out=torch.zeros(6, 31, dtype=torch.int8)),
        lambda: msb.quantize_int8(x.half()),
        lambda: msb.quantize_int8(x, scale=torch.zeros(5)),
        lambda: msb.route(torch.zeros(4, 8), 9),
        lambda: msb.route(torch.zeros(4, 8), 0),
        lambda: msb.route(torch.zeros(4, 8).half(), 2),
        lambda: msb.route(torch.zeros(4, 8), 2, mask=torch.zeros(4)),
        lambda: msb.route(torch.zeros(4, 8), 2, mask=torch.zeros(5, dtype=torch.bool)),
        lambda: msb.route(torch.zeros(4, 8), 2, out=msb.Routing.empty(3, 8, 2, "cpu")),
        lambda: msb.combine(x, msb.Routing(None, torch.zeros(3, 2), None, None, torch.zeros(3, 3, dtype=i32))),
        lambda: msb.combine(x, msb.Routing(None, torch.zeros(3, 2), None, None, torch.zeros(3, 2))),
        lambda: msb.block_norm(x, torch.zeros(5, 32, dtype=bf)),
        lambda: msb.block_norm(x, x, x=torch.zeros(6, 32)),
        lambda: msb.block_norm(x, x, h_out=torch.zeros(6, 32)),
        lambda: msb.block_norm(x, x, gate=torch.zeros(31)),
        lambda: msb.block_norm(x, x, gate=torch.zeros(5, 32)),
        lambda: msb.block_norm(x, x, pre_weight=torch.zeros(31)),
        lambda: msb.block_norm(x, x, pre_weight=torch.zeros(32), post_norm=True, post_weight=torch.zeros(32, dtype=bf)),
    ]
    for i, f in enumerate(cases):
        with pytest.raises(ValueError):
            f()
            pytest.fail("case %d was taken" % i)
    with pytest.raises(ValueError):
        msb.Int8Layer(msb.Dims(64, 16, 2, 1, 0), torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16),
                      torch.zeros(2, 64, 16), torch.zeros(2, 64), torch.zeros(2, 64, dtype=bf))


def test_gate_offsets_pass_32_bits(tmp_path):
    """Offsets of strided gates in 64 bits at every size that the checks admit: the kernels' own
    expression (csrc/dense.h), compiled for the host."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "gate.cpp"
    src.write_text(r"""
#include "dense.h"
int main() {
  msb::NormArgs a = {};
  const int64_t strides[] = {0, 1, 3, 1 << 22, 1 << 23, 1 << 26, (1 << 28) - 1};
  const int rows[] = {0, 1, 255, 256, 16383, 0x7ffffffe};
  for (int64_t row : strides)
    for (int64_t col : strides)
      for (int t : rows)
        for (int i : rows) {
          if (i >= MSB_NORM_MAX_D) continue;
          a.gate_row = row, a.gate_col = col;
          const __int128 want = (__int128)t * row + (__int128)i * col;
          if (a.gate_at(t, i) != want) return 1;
        }
  return 0;
}
""")
    exe = str(tmp_path / "gate")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", os.path.join(root, "include"),
                    "-I", os.path.join(root, "token_top_expert_b200", "csrc"), "-I", "/usr/local/cuda/include",
                    str(src), "-o", exe], check=True)
    subprocess.run([exe], check=True)


def test_row_lengths_have_a_limit(lib, st):
    """Lengths from 2^28 on, whose 32-bit steps along a row would wrap, are refused before any
    launch (one row: its pitch says nothing)."""
    for k in (1 << 28, (1 << 31) - 300, (1 << 31) - 1):
        assert lib.msb_int8_quantize(A, 0, 0, 1, k, B, 0, 2 * B, None) == st.MSB_EUNSUPPORTED
        assert lib.msb_combine(A, 0, 0, 1, B, 2 * B, 1, 1, k, 3 * B, 0, None) == st.MSB_EUNSUPPORTED
        assert lib.msb_combine(A, 0, 0, 1, B, 2 * B, 1, k, 8, 3 * B, 0, None) == st.MSB_EUNSUPPORTED
    # as many (token, run of columns) items as a launch cannot hold
    assert lib.msb_combine(A, 0, 0, 1, B, 2 * B, 1 << 30, 1, 1 << 20, 3 * B, 1 << 20, None) == st.MSB_EUNSUPPORTED


def test_swiglu_int8_has_no_float_output():
    """SwiGLU products are bf16: another out_dtype is refused, as an `out` of another type is."""
    import torch

    import token_top_expert_b200 as msb
    q, w = torch.zeros(6, 32, dtype=torch.int8), torch.zeros(2, 2, 8, 32, dtype=torch.int8)
    offs, qs, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(6), torch.zeros(2, 2, 8)
    for kw in (dict(out_dtype=torch.float32), dict(out_dtype=torch.float16),
               dict(out=torch.zeros(6, 8, dtype=torch.bfloat16), out_dtype=torch.float32), dict(out=torch.zeros(6, 8))):
        with pytest.raises(ValueError, match="SwiGLU|float16|out_dtype"):
            msb.matmul_int8(q, qs, w, ws, offs, swiglu=True, **kw)


def test_int8_linear_scratch_and_out_are_apart(lib, st):
    """out must miss the whole workspace, the rows' scales at its end too."""
    nb = lib.msb_int8_linear_workspace_size(10, 100)
    w = weights(st, stride_n=112)

    def call(out):
        return lib.msb_int8_linear(B, 0, 100, 10, None, None, 1, 10, ctypes.byref(w), A, 64, 100, 0, out, 0, 64,
                                   3 * B, nb, None)
    scales = 3 * B + 10 * 112
    for out in (scales, scales + 36, 3 * B - 64, 3 * B + 4):
        assert call(out) == st.MSB_EINVAL, out - 3 * B


def test_workspaces_lie_in_a_row():
    """A workspace with gaps between its elements is refused: scratch is written byte after byte."""
    import torch

    import token_top_expert_b200 as msb
    gaps = torch.zeros(1 << 16, dtype=torch.uint8)[::2]
    x, w = torch.zeros(6, 32, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.int8)
    for f in (lambda ws: msb.linear_int8(x, w, torch.zeros(8), workspace=ws),
              lambda ws: msb.swiglu_int8(x, w[None].expand(2, 8, 32).contiguous(), torch.zeros(2, 8), workspace=ws),
              lambda ws: msb.route(torch.zeros(4, 8), 2, workspace=ws)):
        with pytest.raises(ValueError, match="contiguous"):
            f(gaps)
