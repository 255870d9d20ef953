"""Host-side checks of the attention side's entry points: bad arguments are
refused before any CUDA call, nothing to do is no error."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attn_ref
import quantized_sparse_moe_router_gb300 as fw


@pytest.fixture(scope="module", autouse=True)
def built():
    fw.build()


def plan(**over):
    a = dict(ctx=4096, new=4096, R=2, page=16, table=4096, blocks=4, free=4096, n_free=8, used=None, T=8, qs=4096, sl=8192,
             req=4096, pos=4096, slot=4096, counts=65536)
    a.update(over)
    return fw.lib().fw_kv_plan(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(R=-1), dict(page=8), dict(page=48), dict(page=0), dict(blocks=0), dict(n_free=-1), dict(T=0),
                                 dict(ctx=None), dict(new=None), dict(table=None), dict(free=None), dict(qs=None), dict(sl=None),
                                 dict(req=None), dict(slot=None), dict(counts=None), dict(ctx=4097), dict(slot=4098),
                                 dict(used=65536), dict(used=65540), dict(R=1 << 21), dict(T=(1 << 30) + 1)])
def test_plan_refuses(bad):
    assert plan(**bad) == fw.FW_EINVAL and fw.fw_moe_last_error()


def rope_args(**over):
    a = dict(T=3, n_q=8, n_kv=2, D=128, rot=128, interleaved=0, eps=1e-6, n_pos=64, q=4096, k=4096, v=4096, q_stride=1024, k_stride=256,
             v_stride=256, q_norm=None, k_norm=None, cos_sin=4096, positions=4096, q_out=4096, k_out=4096, q_out_stride=1024,
             k_out_stride=256, cache=4096, slots=4096, page=16, n_pages=4, status=None)
    a.update(over)
    return fw.FwQkNormRopeArgs(**a)


@pytest.mark.parametrize("bad, status", [
    (dict(D=96), -4), (dict(D=256), -4), (dict(T=-1), -1), (dict(n_q=0), -1), (dict(n_kv=0), -1), (dict(rot=8), -1), (dict(rot=144), -1),
    (dict(interleaved=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(page=24), -1), (dict(n_pages=0), -1),
    (dict(n_pages=1 << 27), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1),
    (dict(q_out=None), -1), (dict(k_out=None, cache=None), -1), (dict(cos_sin=None), -1), (dict(positions=None), -1), (dict(n_pos=0), -1),
    (dict(q_stride=1016), -1), (dict(k_stride=260), -1), (dict(v_stride=128), -1), (dict(k_out_stride=252), -1), (dict(q=4100), -1),
    (dict(cache=4104), -1), (dict(cos_sin=4100), -1), (dict(q_norm=4100), -1), (dict(slots=4098), -1)])
def test_qk_norm_rope_refuses(bad, status):
    assert fw.lib().fw_qk_norm_rope(ctypes.byref(rope_args(**bad)), None) == status and fw.fw_moe_last_error()


def test_qk_norm_rope_nothing_to_do():
    assert fw.lib().fw_qk_norm_rope(ctypes.byref(rope_args(T=0, q=None, k=None, v=None)), None) == fw.FW_OK
    assert fw.lib().fw_qk_norm_rope(None, None) == fw.FW_EINVAL


def attn_args(**over):
    a = dict(R=2, T=8, max_q=4, n_q=8, n_kv=2, D=128, page=16, n_pages=8, max_blocks=4, window=0, sinks=0, scale=0.1, q=4096, out=4096,
             q_stride=1024, out_stride=1024, cache=4096, block_table=4096, q_start=4096, seq_lens=4096, status=None)
    a.update(over)
    return fw.FwAttnQ4Args(**a)


@pytest.mark.parametrize("bad, status", [
    (dict(D=32), -4), (dict(D=96), -4), (dict(n_q=9), -1), (dict(n_q=0), -1), (dict(n_kv=0), -1), (dict(n_q=258), -1), (dict(page=20), -1),
    (dict(n_pages=0), -1), (dict(R=-1), -1), (dict(T=-1), -1), (dict(max_q=-1), -1), (dict(max_q=9), -1), (dict(max_blocks=0), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(scale=0.0), -1), (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1)])
def test_attn_refuses_sizes(bad, status):
    need = ctypes.c_int64(7)
    assert fw.lib().fw_attn_q4_workspace(ctypes.byref(attn_args(**bad)), ctypes.byref(need)) == status
    assert need.value == 0
    assert fw.lib().fw_attn_q4(ctypes.byref(attn_args(**bad)), None, 0, None) == status and fw.fw_moe_last_error()


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=None), dict(cache=None), dict(block_table=None), dict(q_start=None),
                                 dict(seq_lens=None), dict(q=4104), dict(out=4100), dict(cache=4104), dict(block_table=4098),
                                 dict(q_stride=1020), dict(q_stride=512), dict(out_stride=1028), dict(status=4097)])
def test_attn_refuses_pointers(bad):
    assert fw.lib().fw_attn_q4(ctypes.byref(attn_args(**bad)), 65536, 1 << 40, None) == fw.FW_EINVAL and fw.fw_moe_last_error()


def test_attn_nothing_to_do():
    for none in (dict(R=0), dict(T=0, max_q=0), dict(max_q=0)):
        assert fw.lib().fw_attn_q4(ctypes.byref(attn_args(q=None, **none)), None, 0, None) == fw.FW_OK
    assert fw.lib().fw_attn_q4(None, None, 0, None) == fw.FW_EINVAL
    assert fw.lib().fw_attn_q4_workspace(ctypes.byref(attn_args()), None) == fw.FW_EINVAL


@pytest.mark.parametrize("bad, status", [(dict(D=48), -4), (dict(page=8), -1), (dict(T=-1), -1), (dict(cache=None), -1),
                                         (dict(k=4100), -1), (dict(slots=4097), -1), (dict(n_kv=0), -1), (dict(v=None), -1)])
def test_export_refuses(bad, status):
    a = dict(cache=4096, n_pages=4, n_kv=2, D=64, page=16, slots=4096, T=3, k=4096, v=4096, status=None)
    a.update(bad)
    assert fw.lib().fw_kv_export(*a.values(), None) == status and fw.fw_moe_last_error()


def test_structs_match_the_header():
    """ctypes lays the argument structs out as a C compiler does the header's."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [("fw_qk_norm_rope_args", n) for n, _ in fw.FwQkNormRopeArgs._fields_] + [("fw_attn_q4_args", n) for n, _ in fw.FwAttnQ4Args._fields_]
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "fwmoe.h"\nint main(void) {\n'
    src += "".join(f'printf("%zu\\n", offsetof({s}, {n}));\n' for s, n in fields)
    src += 'printf("%zu %zu\\n", sizeof(fw_qk_norm_rope_args), sizeof(fw_attn_q4_args));\nreturn 0; }\n'
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "a.c"), "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), os.path.join(d, "a.c"), "-o", os.path.join(d, "a")], check=True)
        got = subprocess.run([os.path.join(d, "a")], capture_output=True, text=True, check=True).stdout.split()
    by = {"fw_qk_norm_rope_args": fw.FwQkNormRopeArgs, "fw_attn_q4_args": fw.FwAttnQ4Args}
    want = [getattr(by[s], n).offset for s, n in fields] + [ctypes.sizeof(fw.FwQkNormRopeArgs), ctypes.sizeof(fw.FwAttnQ4Args)]
    assert [int(x) for x in got] == want


def test_block_rule_closed_forms():
    """The reference's block rule: extremes, ties and zero blocks."""
    x = np.zeros((4, 32))
    x[0, :4] = [8.0, -8.0, 4.0, 1.5]    # of a tie the positive one sets the scale: d = -1; 8 is exact, -8 clamps to -7
    x[1, :3] = [-16.0, 15.0, 1.0]       # d = 2: 7.5 -> 8 -> clamped to 7, 0.5 -> 0
    x[3, :2] = [0.5, 0.25]
    c, d = attn_ref.quantise(x)
    assert d[:, 0].tolist() == [-1.0, 2.0, 0.0, -0.0625]
    assert attn_ref.values(c, d)[0, 0, :4].tolist() == [8.0, -7.0, 4.0, 2.0]
    assert attn_ref.values(c, d)[1, 0, :3].tolist() == [-16.0, 14.0, 0.0]
    assert (c[2] == 8).all()
    assert attn_ref.values(c, d)[3, 0, :2].tolist() == [0.5, 0.25]


def test_page_format_is_a_bijection():
    """Every nibble of a block's code planes belongs to exactly one (position, dim), and the scales fill the rest."""
    for page in (16, 64):
        for D in (64, 128):
            block = np.zeros(attn_ref.page_bytes(page, D), np.uint8)
            for which in "kv":
                for at in range(page):
                    attn_ref.write_block(block, page, D, at, which, np.full(D, 15), np.full(D // 32, 0xFFFF))
            assert (block == 255).all()
