"""include/ssu_delta.h and include/ssu_verify.h without a GPU: exports, struct
layout as a C compiler sees it, refusals before any launch.  The pointers are
never dereferenced."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch  # noqa: F401  (before the library, which then shares torch's HIP runtime instead of loading a second one)

import speculative_replay_state_amd as ssu
from speculative_replay_state_amd import delta, verification

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned


@pytest.mark.parametrize("header,module", [("ssu_delta.h", delta), ("ssu_verify.h", verification)])
def test_exports_every_declared_symbol(header, module):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(ssu_[a-z_]+)\s*\(", src))
    assert names == set(module.EXPORTED)
    lib = ctypes.CDLL(ssu.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_struct_layouts_and_constants_match_ctypes(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    structs = (("ssu_delta_cache", ssu.SsuDeltaCache), ("ssu_delta_step", ssu.SsuDeltaStep),
               ("ssu_delta_prefill_args", ssu.SsuDeltaPrefill), ("ssu_verify_args", ssu.SsuVerify))
    consts = ("SSU_DELTA_MAX_PAIRS", "SSU_STATUS_BAD_TOKEN", "SSU_STATUS_BAD_PROBS")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ssu_delta.h"', '#include "ssu_verify.h"', 'int main(void) {']
    for cname, ctype in structs:
        lines.append('  printf("%s %%zu\\n", sizeof(%s));' % (cname, cname))
        lines += ['  printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (cname, f, cname, f) for f, _ in ctype._fields_]
    lines += ['  printf("%s %%zu\\n", (size_t)(%s));' % (c, c) for c in consts] + ['  return 0;', '}']
    (tmp_path / "a.c").write_text("\n".join(lines) + "\n")
    subprocess.run([gcc, "-std=c11", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", str(tmp_path / "a.c"), "-o", str(tmp_path / "a")], check=True)
    out = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout
    got = {k: int(v) for k, v in (line.split() for line in out.splitlines())}
    for cname, ctype in structs:
        assert got[cname] == ctypes.sizeof(ctype), cname
        for f, _ in ctype._fields_:
            assert got["%s.%s" % (cname, f)] == getattr(ctype, f).offset, (cname, f)
    for c in consts:
        assert got[c] == getattr(ssu, c), c


def _fill(struct, base, kw):
    for k, v in {**base, **kw}.items():
        setattr(struct, k, v)
    return struct


def _cache(**kw):
    return _fill(ssu.SsuDeltaCache(), dict(
        num_slots=8, nheads_k=2, nheads_v=4, dim_k=128, dim_v=128, ring_len=16, state_dtype=ssu.SSU_BF16,
        io_dtype=ssu.SSU_BF16, state=FAKE, state_slot_stride=4 * 128 * 128 * 2, k_cache=FAKE, k_slot_stride=2 * 16 * 256,
        v_cache=FAKE, v_slot_stride=4 * 16 * 256, gate_cache=FAKE, gate_slot_stride=4 * 16 * 8, ring_start=FAKE), kw)


INPUTS = dict(q=FAKE, k=FAKE, v=FAKE, q_row_stride=256, k_row_stride=256, v_row_stride=512, dt=FAKE, beta=FAKE, A=FAKE,
              dt_bias=FAKE, scale=1.0, out=FAKE, out_dtype=ssu.SSU_BF16)


def _step(**kw):
    return _fill(ssu.SsuDeltaStep(), dict(batch=3, max_seqlen=4, slot_idx=FAKE, prev_num_accepted=FAKE, **INPUTS), kw)


def _prefill(**kw):
    return _fill(ssu.SsuDeltaPrefill(), dict(num_seqs=2, rows=70, nheads_k=2, nheads_v=4, dim_k=128, dim_v=128,
                                             io_dtype=ssu.SSU_BF16, cu_seqlens=FAKE, workspace=FAKE,
                                             workspace_bytes=1 << 30, **INPUTS), kw)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(num_slots=0), -1, "num_slots"),
    (dict(nheads_k=0), -1, "positive"),
    (dict(nheads_v=-4), -1, "positive"),
    (dict(nheads_v=3), -1, "multiple"),
    (dict(dim_k=96), -2, "dim_k"),
    (dict(dim_v=8), -2, "dim_v"),
    (dict(dim_v=24), -2, "dim_v"),
    (dict(dim_v=272), -2, "dim_v"),
    (dict(nheads_v=1 << 16), -2, "2^23"),
    (dict(ring_len=0), -2, "ring_len"),
    (dict(ring_len=33), -2, "ring_len"),
    (dict(state_dtype=ssu.SSU_FP8_E4M3), -2, "state_dtype"),
    (dict(state_dtype=77), -1, "state_dtype"),
    (dict(io_dtype=ssu.SSU_F16), -2, "io_dtype"),
    (dict(state=None), -1, "NULL"),
    (dict(gate_cache=None), -1, "NULL"),
    (dict(k_cache=FAKE + 8), -1, "aligned"),
    (dict(ring_start=FAKE + 2), -1, "aligned"),
    (dict(state_slot_stride=4 * 128 * 128 * 2 - 16), -1, "state slot stride"),
    (dict(v_slot_stride=4 * 16 * 256 + 8), -1, "multiple of 16"),
    (dict(gate_slot_stride=16), -1, "gate_cache slot stride"),
    (dict(gate_slot_stride=4 * 16 * 8 + 4), -1, "multiple of 8"),
    (dict(gate_cache=FAKE + 4), -1, "aligned"),
])
def test_cache_refusals(kw, code, msg):
    c = _cache(**kw)
    for rc in (ssu.delta.ssu_delta_replay_step(c, _step()), delta.ssu_delta_flush(c, FAKE, FAKE, 3),
               delta.ssu_delta_init_state(c, FAKE, 0, FAKE, 3), delta.ssu_delta_read_state(c, FAKE, 1 << 20, FAKE, 3)):
        assert rc == code
        assert msg in ssu.ssu_last_error()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(batch=-1), -1, "batch"),
    (dict(batch=1 << 20), -2, "SSU_DELTA_MAX_PAIRS"),
    (dict(max_seqlen=0), -1, "max_seqlen"),
    (dict(max_seqlen=17), -1, "max_seqlen"),
    (dict(slot_idx=None), -1, "NULL"),
    (dict(prev_num_accepted=FAKE + 1), -1, "aligned"),
    (dict(q=None), -1, "NULL"),
    (dict(A=None), -1, "NULL"),
    (dict(v=FAKE + 8), -1, "aligned"),
    (dict(beta=FAKE + 2), -1, "aligned"),
    (dict(q_row_stride=248), -1, "q_row_stride"),
    (dict(v_row_stride=516), -1, "v_row_stride"),
    (dict(out_dtype=ssu.SSU_F16), -2, "out_dtype"),
])
def test_step_refusals(kw, code, msg):
    assert delta.ssu_delta_replay_step(_cache(), _step(**kw)) == code
    assert msg in ssu.ssu_last_error()


def test_step_longer_than_16_tokens_is_unsupported():
    c = _cache(ring_len=32, k_slot_stride=2 * 32 * 256, v_slot_stride=4 * 32 * 256, gate_slot_stride=4 * 32 * 8)
    assert delta.ssu_delta_replay_step(c, _step(max_seqlen=17)) == ssu.SSU_ERR_UNSUPPORTED


def test_empty_calls_are_no_ops():
    assert delta.ssu_delta_replay_step(_cache(), _step(batch=0, q=None)) == 0
    assert delta.ssu_delta_flush(_cache(), None, None, 0) == 0
    assert delta.ssu_delta_init_state(_cache(), None, 0, None, 0) == 0
    assert delta.ssu_delta_prefill(_prefill(num_seqs=0, cu_seqlens=None)) == 0
    assert ssu.ssu_last_error() == ""


@pytest.mark.parametrize("stride,read,msg", [(-4, False, "stride"), (6, False, "stride"), (4, False, "packed"),
                                             (0, True, "packed"), (65536 - 4, True, "packed")])
def test_state_stride_refusals(stride, read, msg):
    fn = delta.ssu_delta_read_state if read else delta.ssu_delta_init_state
    assert fn(_cache(), FAKE, stride, FAKE, 2) == ssu.SSU_ERR_INVALID
    assert msg in ssu.ssu_last_error()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(num_seqs=-1), -1, "num_seqs"),
    (dict(num_seqs=1 << 21), -2, "SSU_DELTA_MAX_PAIRS"),
    (dict(rows=-1), -1, "rows"),
    (dict(rows=(1 << 28) + 1), -2, "2^30"),
    (dict(dim_k=32), -2, "dim_k"),
    (dict(nheads_v=5), -1, "multiple"),
    (dict(io_dtype=ssu.SSU_F32), -2, "io_dtype"),
    (dict(cu_seqlens=None), -1, "cu_seqlens"),
    (dict(initial_states=FAKE + 4), -1, "initial_states"),
    (dict(k=None), -1, "NULL"),
    (dict(k_row_stride=128), -1, "k_row_stride"),
    (dict(q_row_stride=1 << 23), -2, "2^23"),
    (dict(nheads_v=1 << 16, rows=0, num_seqs=1), -2, "2^23"),
    (dict(workspace=None), -4, "workspace"),
    (dict(workspace_bytes=64), -4, "workspace"),
    (dict(workspace=FAKE + 4), -1, "workspace"),
    (dict(out_dtype=9), -2, "out_dtype"),
])
def test_prefill_refusals(kw, code, msg):
    assert delta.ssu_delta_prefill(_prefill(**kw)) == code
    assert msg in ssu.ssu_last_error()


def test_prefill_workspace_size():
    size = ssu.delta_prefill_workspace_size
    assert size(0, 1, 1) > 0 and size(64, 1, 4) == 3 * size(0, 1, 4)
    assert size(-1, 1, 1) == 0 and "rows" in ssu.ssu_last_error()
    assert size(1, -1, 1) == 0 and size(1, 1, 0) == 0


def _verify(**kw):
    return _fill(ssu.SsuVerify(), dict(
        batch=3, max_seqlen=4, vocab=1000, ring_len=16, probs_dtype=ssu.SSU_F32, tokens=FAKE, target_probs=FAKE,
        target_row_stride=1000, draft_probs=FAKE, draft_row_stride=1000, u=FAKE, u_final=FAKE, out_tokens=FAKE,
        num_accepted=FAKE, live=FAKE, next_live=FAKE, workspace=FAKE, workspace_bytes=1 << 20), kw)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(batch=-1), -1, "batch"),
    (dict(batch=65536), -2, "batch"),
    (dict(vocab=0), -1, "vocab"),
    (dict(vocab=(1 << 24) + 1), -2, "vocab"),
    (dict(batch=60000, vocab=1 << 22), -2, "2^23"),
    (dict(max_seqlen=0), -1, "max_seqlen"),
    (dict(max_seqlen=65), -2, "max_seqlen"),
    (dict(probs_dtype=ssu.SSU_FP8_E4M3), -2, "probs_dtype"),
    (dict(tokens=None), -1, "NULL"),
    (dict(u_final=None), -1, "NULL"),
    (dict(target_row_stride=999), -1, "stride"),
    (dict(draft_row_stride=0), -1, "stride"),
    (dict(target_probs=FAKE + 2), -1, "aligned"),
    (dict(next_fold=FAKE + 2), -1, "aligned"),
    (dict(live=None), -1, "live"),
    (dict(ring_len=3), -1, "ring_len"),
    (dict(reserve=17), -1, "reserve"),
    (dict(reserve=-1), -1, "reserve"),
    (dict(next_live=None, next_left=FAKE), -1, "next_live"),
    (dict(workspace=None), -4, "workspace"),
    (dict(workspace_bytes=8), -4, "workspace"),
    (dict(workspace=FAKE + 8), -1, "workspace"),
])
def test_verify_refusals(kw, code, msg):
    assert verification.ssu_verify(_verify(**kw)) == code
    assert msg in ssu.ssu_last_error()


def test_verify_no_op_and_workspace():
    assert verification.ssu_verify(_verify(batch=0, tokens=None)) == 0
    assert ssu.verify_workspace_size(3, 4096) == 3 * (4 + 2) * 8 and ssu.verify_workspace_size(3, 4097) == 3 * (5 + 2) * 8
    assert ssu.verify_workspace_size(-1, 5) == 0


def test_front_end_refuses_host_tensors():
    import torch
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        ssu.DeltaCache(2, 1, 1, 4, "bf16", z(2, 1 << 14), z(2, 1 << 10), z(2, 1 << 10), z(2, 1 << 10), z(2, dt=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        ssu.make_delta_prefill(z(2, dt=torch.int32), z(4, 1, 64), z(4, 1, 64), z(4, 1, 64), z(4, 1), z(4, 1), z(1), z(1), z(4, 1, 64))
    with pytest.raises(ValueError, match="device tensor"):
        ssu.make_verify(z(4, dt=torch.int32), z(4, 9), None, z(4), z(1), z(1, 4, dt=torch.int32), z(1, dt=torch.int32), z(8))


def test_expanded_probability_rows_are_refused(monkeypatch):
    """One row expanded over several has no distance between rows; only a single row needs none."""
    import torch
    from speculative_replay_state_amd import verification as V
    monkeypatch.setattr(V, "_on_device", lambda t, name: None)
    row = torch.zeros(1, 10)
    assert V._probs(row, "p", 1, 10) == 10 and V._probs(torch.zeros(3, 16)[:, :10], "p", 3, 10) == 16
    for t in (row.expand(3, -1), torch.zeros(40).as_strided((3, 10), (4, 1))):
        with pytest.raises(ValueError, match="target_probs: its rows overlap"):
            V._probs(t, "target_probs", 3, 10)
