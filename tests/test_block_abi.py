"""The decoder-block operators without a GPU: declared, exported and laid out as the header
says, and refusing bad arguments with the documented status before launching anything."""
import ctypes
import math
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "awq_block.h")

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")
block = pytest.importorskip("bit_weight_only_w4a16_amd.block")

import block_ctypes as c_abi  # noqa: E402

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
    assert names == sorted(block.EXPORTS) == sorted(c_abi._SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


def test_structures_match_the_header(tmp_path):
    """Sizes and offsets as a C compiler lays out the header's structures."""
    pairs = {"awq_rope_args": c_abi.RopeArgs, "awq_attn_prompt_args": c_abi.AttnPromptArgs,
             "awq_attn_tree_args": c_abi.AttnTreeArgs, "awq_epilogue": c_abi.Epilogue}
    lines = []
    for c, py in pairs.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f[0]} %zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "awq_block.h"\nint main(void) {' + "\n".join(lines) + "return 0; }")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(rocm, "include"), str(src), "-o", exe], check=True)
    got = dict(line.rsplit(" ", 1) for line in subprocess.run([exe], capture_output=True, text=True,
                                                             check=True).stdout.splitlines())
    for c, py in pairs.items():
        assert int(got[c]) == ctypes.sizeof(py)
        for f in py._fields_:
            assert int(got[f"{c}.{f[0]}"]) == getattr(py, f[0]).offset, f"{c}.{f[0]}"


def call(fn, args):
    return fn(ctypes.byref(args), None)


ROPE = dict(q=P, q_out=P, k=P, k_out=None, v=P, k_cache=P, v_cache=P, positions=P, inv_freq=P, slots=P, tokens=4,
            q_token=512, q_head=128, qo_token=512, qo_head=128, k_token=256, k_head=128, v_token=256, v_head=128,
            cache_page=4096, cache_head=2048, cache_slot=128, pages=8, page_size=16, q_heads=4, kv_heads=2,
            head_dim=128, rot_dim=128, dtype=0, scale=1.0)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0), OK), (dict(tokens=0, q=None), OK), (dict(tokens=-1), INVALID), (dict(reserved=1), INVALID),
    (dict(q=None, k=None), INVALID), (dict(q_out=None), INVALID), (dict(k=None), INVALID),
    (dict(k_cache=None, v_cache=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID), (dict(dtype=2), INVALID),
    (dict(head_dim=100), INVALID), (dict(rot_dim=130), INVALID), (dict(rot_dim=3), INVALID),
    (dict(rot_dim=-2), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(cache_slot=64), INVALID), (dict(q_token=64), INVALID),
    (dict(q_head=64), INVALID), (dict(k_token=-8), INVALID), (dict(head_dim=136, rot_dim=8), UNSUPPORTED),
    (dict(q_token=1 << 23), UNSUPPORTED), (dict(tokens=(1 << 30) + 1), UNSUPPORTED), (dict(q=P + 8), MISALIGNED),
    (dict(k_cache=P + 2), MISALIGNED), (dict(q_token=516), MISALIGNED), (dict(cache_page=4100), MISALIGNED),
    (dict(positions=P + 2), MISALIGNED), (dict(slots=P + 4), MISALIGNED),
])
def test_rope_refusals(lib, change, code):
    assert call(lib.awq_rope, c_abi.RopeArgs(**{**ROPE, **change})) == code


PROMPT = dict(q=P, k=P, v=P, out=P, cu=P, tokens=100, seqs=2, q_token=512, q_head=128, k_token=256, k_head=128,
              v_token=256, v_head=128, o_token=512, o_head=128, q_heads=4, kv_heads=2, head_dim=128, dtype=0, scale=0.1)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0, q=None), OK), (dict(seqs=0), OK), (dict(tokens=-1), INVALID), (dict(seqs=-1), INVALID),
    (dict(reserved=1), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(cu=None), INVALID), (dict(q_heads=3), INVALID), (dict(kv_heads=0), INVALID),
    (dict(dtype=-1), INVALID), (dict(head_dim=60), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(k_token=120), INVALID), (dict(v_head=-8), INVALID),
    (dict(head_dim=256), UNSUPPORTED), (dict(k_token=1 << 23), UNSUPPORTED), (dict(q_heads=8192), UNSUPPORTED),
    (dict(tokens=1 << 30, q_heads=4096, seqs=1), UNSUPPORTED), (dict(q=P + 8), MISALIGNED),
    (dict(tokens=1 << 29, seqs=1 << 22), UNSUPPORTED),
    (dict(out=P + 4), MISALIGNED), (dict(cu=P + 2), MISALIGNED), (dict(k_head=132), MISALIGNED),
])
def test_prompt_refusals(lib, change, code):
    assert call(lib.awq_attn_prompt, c_abi.AttnPromptArgs(**{**PROMPT, **change})) == code


TREE = dict(q=P, k_cache=P, v_cache=P, out=P, block_table=P, ctx_lens=P, cu_q=P, mask=P, ws=P, ws_bytes=1 << 40,
            tokens=8, seqs=2, table_width=64, pages=100, q_token=512, q_head=128, o_token=512, o_head=128,
            cache_page=4096, cache_head=2048, cache_slot=128, page_size=16, max_q=4, q_heads=4, kv_heads=2,
            head_dim=128, dtype=0, scale=0.1)


@pytest.mark.parametrize("change,code", [
    (dict(tokens=0, q=None), OK), (dict(seqs=0), OK), (dict(tokens=-1), INVALID), (dict(reserved=1), INVALID),
    (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(out=None), INVALID),
    (dict(block_table=None), INVALID), (dict(ctx_lens=None), INVALID), (dict(cu_q=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws=None, ws_bytes=0), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(max_q=0), INVALID), (dict(max_q=65), UNSUPPORTED), (dict(table_width=0), INVALID),
    (dict(page_size=0), INVALID), (dict(pages=0), INVALID), (dict(q_heads=5), INVALID), (dict(dtype=7), INVALID),
    (dict(scale=0.0), INVALID), (dict(seqs=65536), UNSUPPORTED), (dict(head_dim=136), UNSUPPORTED),
    (dict(table_width=1 << 27), UNSUPPORTED), (dict(cache_slot=120), INVALID), (dict(cache_head=-8), INVALID),
    (dict(q=P + 2), MISALIGNED), (dict(mask=P + 4), MISALIGNED), (dict(ws=P + 8), MISALIGNED),
    (dict(cache_head=2044), MISALIGNED), (dict(ctx_lens=P + 1), MISALIGNED),
    (dict(tokens=1 << 30), UNSUPPORTED),
])
def test_tree_refusals(lib, change, code):
    assert call(lib.awq_attn_tree, c_abi.AttnTreeArgs(**{**TREE, **change})) == code


def test_tree_workspace_sizes(lib):
    f = block.awq_attn_tree_workspace_bytes
    assert f(0, 2, 64, 16, 4, 4, 2, 128) == 0
    assert f(8, 2, 64, 16, 65, 4, 2, 128) == 0                  # refused
    assert f(8, 2, 4, 16, 4, 4, 2, 128) == 0                     # 64 positions: one split
    # per token, head and split: a row of D sums, a maximum and a sum
    assert f(8, 2, 64, 16, 4, 4, 2, 128) % (8 * 4 * 130 * 4) == 0
    assert f(8, 2, 64, 16, 4, 4, 2, 128) > 0


@pytest.mark.parametrize("change,code", [
    (dict(), OK), (dict(epi=None), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(reserved=1), INVALID), (dict(bias=P + 2), MISALIGNED), (dict(mul=P + 8), MISALIGNED),
    (dict(residual=P + 4), MISALIGNED), (dict(n=100), INVALID), (dict(m=-1), INVALID), (dict(x=P + 2), MISALIGNED),
    (dict(group=96, k=384), UNSUPPORTED),
])
def test_fused_refusals(lib, change, code):
    d = dict(m=0, n=128, k=256, group=128, x=P, act=0, reserved=0, bias=None, mul=None, residual=None, epi=True)
    d.update(change)
    e = c_abi.Epilogue(d["bias"], d["mul"], d["residual"], d["act"], d["reserved"])
    rc = lib.awq_gemm_fused(d["x"], None, P, d["m"], d["n"], d["k"], d["group"], 0,
                            ctypes.byref(e) if d["epi"] else None, P, None, 0, None)
    assert rc == code


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        block.awq_attn_prompt(x, x, x, cu)
    with pytest.raises(ValueError):
        block.awq_rope(x, cu, torch.ones(4))
    with pytest.raises(ValueError):
        block.awq_rope(None, cu, torch.ones(4))
    with pytest.raises(ValueError):
        block.awq_attn_tree(x, x[None], x[None], cu[None], cu[:1], cu, 1)
    with pytest.raises(ValueError):
        block.awq_gemm_fused(x[0], None, x[0], 128, 64, act="tanh")
    with pytest.raises(ValueError):
        block.awq_gemm_fused(x[0], None, x[0], 128, 128)
    with pytest.raises(TypeError):
        block.awq_attn_prompt([1.0], x, x, cu)
    with pytest.raises(TypeError):
        block.awq_rope(x, None, None)


def test_rope_frequencies():
    base, one = block.rope_frequencies(64)
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert one == 1.0 and torch.allclose(base.double(), torch.tensor(want, dtype=torch.float64), rtol=1e-7)
    linear, _ = block.rope_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(linear, base / 4)
    ntk, _ = block.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(base[-1]) / 4, rel_tol=1e-6)
    for name in ("bands", "yarn"):
        f, s = block.rope_frequencies(64, scaling=name, factor=8.0, original=4096, low=1.0, high=32.0)
        ratio = base / f
        assert ratio[0] == 1.0 and math.isclose(float(ratio[-1]), 8.0, rel_tol=1e-6)
        assert bool((ratio[1:] >= ratio[:-1] - 1e-6).all())
        assert s == (1.0 if name == "bands" else pytest.approx(0.1 * math.log(8.0) + 1))
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, scaling="cubic"), dict(rot_dim=8, factor=0.5),
                dict(rot_dim=2, scaling="ntk"), dict(rot_dim=8, scaling="yarn", low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            block.rope_frequencies(**bad)


def test_tree_mask():
    m = block.tree_mask([-1, 0, 0, 1, -1])
    assert m.tolist() == [1, 3, 5, 11, 16]
    chain = block.tree_mask(range(-1, 63))
    assert chain[-1].item() == -1 and chain[62].item() == (1 << 63) - 1
    for bad in ([0], [-1, 1], [-2], range(-1, 64)):
        with pytest.raises(ValueError):
            block.tree_mask(bad)
