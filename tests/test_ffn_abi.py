"""The feed-forward operators without a GPU: declared, exported and laid out as the header says,
and refusing bad arguments with the documented status before launching anything."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "awq_ffn.h")

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
int8 = pytest.importorskip("bit_weight_only_w4a16_amd.int8")
moe = pytest.importorskip("bit_weight_only_w4a16_amd.moe")

import ffn_ctypes as c_abi  # noqa: E402

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20   # an aligned stand-in address; never dereferenced, because validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(awq.LIB_PATH):
        pytest.skip("library not built")
    return c_abi.lib()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(awq_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(int8.EXPORTS + moe.EXPORTS) == sorted(c_abi._SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


def test_structures_match_the_header(tmp_path):
    lines = []
    for c, py in c_abi.STRUCTS.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f[0]} %zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "awq_ffn.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(rocm, "include"), str(src), "-o", exe], check=True)
    got = dict(line.rsplit(" ", 1) for line in subprocess.run([exe], capture_output=True, text=True,
                                                             check=True).stdout.splitlines())
    for c, py in c_abi.STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f in py._fields_:
            assert int(got[f"{c}.{f[0]}"]) == getattr(py, f[0]).offset, f"{c}.{f[0]}"


def call(fn, args):
    return fn(ctypes.byref(args), None)


NORM = dict(x=P, residual=P, weight=P, h_out=P, y=P, q=P, scale=P, tokens=4, x_stride=256, residual_stride=256,
            h_stride=256, y_stride=256, q_stride=256, width=256, dtype=0, eps=1e-5)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0), OK), (dict(tokens=0, x=None), OK), (dict(tokens=-1), INVALID), (dict(reserved=1), INVALID),
    (dict(x=None), INVALID), (dict(y=None, q=None, scale=None), INVALID), (dict(scale=None), INVALID),
    (dict(q=None), INVALID), (dict(residual=None), INVALID), (dict(width=0), INVALID), (dict(width=252), INVALID),
    (dict(dtype=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x_stride=248), INVALID), (dict(q_stride=248), INVALID),
    (dict(width=32776, x_stride=1 << 20), UNSUPPORTED), (dict(tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(x=P + 8), MISALIGNED), (dict(weight=P + 2), MISALIGNED), (dict(scale=P + 2), MISALIGNED),
    (dict(y_stride=260), MISALIGNED), (dict(q=P + 8), MISALIGNED), (dict(h_stride=1 << 31), UNSUPPORTED),
])
def test_rms_norm_refusals(lib, change, code):
    assert call(lib.awq_rms_norm, c_abi.RmsNormArgs(**{**NORM, **change})) == code


QUANT = dict(x=P, inv_s_c=P, q=P, scale=P, tokens=4, x_stride=256, q_stride=256, width=256, dtype=1)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0), OK), (dict(tokens=-1), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID),
    (dict(scale=None), INVALID), (dict(width=12), INVALID), (dict(dtype=-1), INVALID), (dict(x_stride=0), INVALID),
    (dict(inv_s_c=P + 8), MISALIGNED), (dict(q_stride=257), MISALIGNED), (dict(width=65536, x_stride=65536, q_stride=65536),
                                                                       UNSUPPORTED),
])
def test_quant_refusals(lib, change, code):
    assert call(lib.awq_quant_i8, c_abi.QuantI8Args(**{**QUANT, **change})) == code


def test_packed_sizes(lib):
    f = int8.awq_packed_i8_bytes
    assert f(16, 64) == 1024 + 256          # one unit, 16 scales, rounded up to 256
    assert f(24, 80) == 2 * 2 * 1024 + 256  # rows to 32, channels to 128
    assert f(12, 64) == f(16, 24) == f(0, 64) == f(16, -16) == f(16, 131072) == f(1 << 20, 1 << 12) == 0
    assert f(1 << 20, 1024) > 0


@pytest.mark.parametrize("change,code", [
    (dict(n=12), INVALID), (dict(k=24), INVALID), (dict(dtype=3), INVALID), (dict(w=None), INVALID),
    (dict(packed=None), INVALID), (dict(k=131072), UNSUPPORTED), (dict(n=1 << 20, k=2048), UNSUPPORTED),
    (dict(w=P + 8), MISALIGNED), (dict(s_c=P + 2), MISALIGNED), (dict(bytes=1024), WORKSPACE),
])
def test_pack_refusals(lib, change, code):
    d = {**dict(w=P, s_c=P, n=16, k=64, dtype=0, packed=P, bytes=1280), **change}
    assert lib.awq_pack_i8(d["w"], d["s_c"], d["n"], d["k"], d["dtype"], d["packed"], d["bytes"], None) == code


GEMM = dict(q=P, scale=P, packed=P, bias=P, mul=P, residual=P, y=P, ws=P, ws_bytes=1 << 40, M=4, N=64, K=64,
            q_stride=64, dtype=0, act=0)


@pytest.mark.parametrize("change,code", [
    (dict(M=0, q=None), OK), (dict(M=-1), INVALID), (dict(N=60), INVALID), (dict(K=72), INVALID), (dict(act=5), INVALID),
    (dict(act=-1), INVALID), (dict(dtype=2), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(packed=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(q_stride=48), INVALID),
    (dict(K=131072, q_stride=131072), UNSUPPORTED), (dict(q_stride=1 << 23), UNSUPPORTED),
    (dict(M=1 << 30), UNSUPPORTED), (dict(M=1 << 24, N=1 << 12), UNSUPPORTED), (dict(q_stride=72), MISALIGNED),
    (dict(q=P + 8), MISALIGNED), (dict(scale=P + 1), MISALIGNED), (dict(bias=P + 4), MISALIGNED),
    (dict(ws=P + 8), MISALIGNED), (dict(mul=P + 2), MISALIGNED),
])
def test_gemm_i8_refusals(lib, change, code):
    assert call(lib.awq_gemm_i8, c_abi.GemmI8Args(**{**GEMM, **change})) == code


def test_gemm_i8_asks_for_its_workspace(lib):
    """Every size whose workspace is not empty is refused with less."""
    f = int8.awq_gemm_i8_workspace_bytes
    assert f(0, 64, 64) == f(4, 60, 64) == f(4, 64, 131072) == 0
    for m, n, k in [(1, 256, 14336), (100, 512, 8192), (300, 4096, 11008), (2000, 256, 16384)]:
        need = f(m, n, k)
        d = {**GEMM, "M": m, "N": n, "K": k, "q_stride": k, "ws_bytes": max(need - 1, 0)}
        if need:
            assert call(lib.awq_gemm_i8, c_abi.GemmI8Args(**d)) == WORKSPACE
            assert call(lib.awq_gemm_i8, c_abi.GemmI8Args(**{**d, "ws": None, "ws_bytes": 0})) == WORKSPACE


ROUTE = dict(x=P, w=P, bias=P, ids=P, weights=P, ws=P, ws_bytes=1 << 40, tokens=40, x_stride=256, hidden=256, experts=16,
             k=2, dtype=0, score=0, renormalize=1, scale=1.0)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0, x=None), OK), (dict(tokens=-1), INVALID), (dict(reserved=1), INVALID), (dict(hidden=252), INVALID),
    (dict(experts=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(dtype=2), INVALID),
    (dict(score=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(ws=None), INVALID), (dict(x_stride=248), INVALID),
    (dict(ws=None, ws_bytes=0), WORKSPACE), (dict(ws_bytes=16), WORKSPACE), (dict(experts=1025), UNSUPPORTED),
    (dict(experts=64, k=33), UNSUPPORTED), (dict(tokens=(1 << 20) + 1), UNSUPPORTED),
    (dict(hidden=65544, x_stride=65544), UNSUPPORTED), (dict(w=P + 8), MISALIGNED), (dict(ids=P + 2), MISALIGNED),
    (dict(x_stride=260), MISALIGNED), (dict(ws=P + 8), MISALIGNED),
])
def test_route_refusals(lib, change, code):
    assert call(lib.awq_moe_route, c_abi.MoeRouteArgs(**{**ROUTE, **change})) == code


def test_route_workspace_sizes(lib):
    f = moe.awq_moe_route_workspace_bytes
    assert f(0, 256, 16) == f(-1, 256, 16) == f(4, 252, 16) == f(4, 256, 2000) == 0
    assert f(4, 4096, 16) == 0 and f(5, 4096, 16) > 0 and f(4, 4104, 16) > 0 and f(1, 8, 65) > 0
    # a float64 for each token and expert, of each slice of the channels
    assert f(517, 4096, 128) % (517 * 128 * 8) == 0


MOE = dict(x=P, ids=P, weights=P, gate=P, up=P, down=P, inv_in=P, inv_down=P, residual=P, y=P, ws=P, ws_bytes=1 << 40,
           tokens=4, x_stride=256, residual_stride=256, y_stride=256, inv_in_stride=256, inv_down_stride=384, hidden=256,
           ffn=384, experts=8, k=2, group=128, fmt=0, act=4)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0, x=None), OK), (dict(tokens=-1), INVALID), (dict(tokens=65), UNSUPPORTED), (dict(reserved=1), INVALID),
    (dict(hidden=0), INVALID), (dict(ffn=-128), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED),
    (dict(experts=0), INVALID), (dict(experts=1025), UNSUPPORTED), (dict(fmt=2), INVALID), (dict(act=5), INVALID),
    (dict(group=0), INVALID), (dict(group=256), INVALID), (dict(group=96), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(hidden=320, x_stride=320, residual_stride=320, y_stride=320, group=64), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(gate=None), INVALID), (dict(up=None), INVALID),
    (dict(down=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=64), WORKSPACE),
    (dict(ws=None, ws_bytes=0), WORKSPACE), (dict(x_stride=248), INVALID), (dict(y_stride=260), MISALIGNED),
    (dict(inv_in_stride=128), INVALID), (dict(inv_down_stride=128), INVALID), (dict(gate=P + 8), MISALIGNED),
    (dict(ids=P + 2), MISALIGNED), (dict(inv_down=P + 2), MISALIGNED),
    (dict(hidden=1 << 17, ffn=1 << 14, x_stride=1 << 17), UNSUPPORTED),
])
def test_moe_refusals(lib, change, code):
    assert call(lib.awq_moe, c_abi.MoeArgs(**{**MOE, **change})) == code


def test_null_structures(lib):
    for name in ("awq_rms_norm", "awq_quant_i8", "awq_gemm_i8", "awq_moe_route", "awq_moe"):
        assert getattr(lib, name)(None, None) == INVALID


def test_binding_refuses_host_tensors_and_unknown_names():
    x = torch.zeros(2, 64, dtype=torch.float16)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    for f in (lambda: int8.awq_rms_norm(x), lambda: int8.awq_quant_i8(x), lambda: int8.awq_pack_i8(x),
              lambda: int8.awq_gemm_i8(x.to(torch.int8), x[0].float(), x, 16, 64),
              lambda: int8.awq_gemm_i8(x, x, x, 16, 64, act="tanh"), lambda: moe.awq_moe_route(x, x, 1),
              lambda: moe.awq_moe_route(x, x, 1, score="topk"), lambda: moe.awq_moe(x, ids, x, x, x, x, 128, act="tanh"),
              lambda: moe.awq_moe(x, ids, ids, x, x, x, 128)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: int8.awq_gemm_i8(x, x, x, 16, 64, dtype=torch.float32), lambda: int8.awq_rms_norm([1.0]),
              lambda: moe.awq_moe_route(None, x, 1)):
        with pytest.raises(TypeError):
            f()
