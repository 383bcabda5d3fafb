"""include/ssu_prefill.h and include/ssu_logits.h without a GPU: exports, struct
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
from speculative_replay_state_amd import prompts, sampling

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned
INVALID, UNSUPPORTED, WORKSPACE = ssu.SSU_ERR_INVALID, ssu.SSU_ERR_UNSUPPORTED, ssu.SSU_ERR_WORKSPACE


@pytest.mark.parametrize("header,module", [("ssu_prefill.h", prompts), ("ssu_logits.h", sampling)])
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
    structs = (("ssu_prefill_args", ssu.SsuPrefill), ("ssu_history", ssu.SsuHistory), ("ssu_count_args", ssu.SsuCount),
               ("ssu_logits_args", ssu.SsuLogits))
    consts = ("SSU_STATUS_EMPTY_ROW", "SSU_STATUS_BAD_BIAS")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ssu_prefill.h"', '#include "ssu_logits.h"', 'int main(void) {']
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


def _prefill(**kw):
    return _fill(ssu.SsuPrefill(), dict(
        num_seqs=2, rows=70, nheads=4, ngroups=2, headdim=64, dstate=128, io_dtype=ssu.SSU_BF16, out_dtype=ssu.SSU_BF16,
        cu_seqlens=FAKE, x=FAKE, B=FAKE, C=FAKE, x_row_stride=256, B_row_stride=256, C_row_stride=256, dt=FAKE, A=FAKE, D=FAKE,
        dt_bias=FAKE, out=FAKE, workspace=FAKE, workspace_bytes=1 << 30), kw)


def _refused(rc, code, words):
    assert rc == code, (rc, ssu.ssu_last_error())
    assert words in ssu.ssu_last_error(), ssu.ssu_last_error()


@pytest.mark.parametrize("kw,code,words", [
    (dict(num_seqs=-1), INVALID, "num_seqs"), (dict(rows=-1), INVALID, "rows"), (dict(nheads=0), INVALID, "nheads"),
    (dict(ngroups=0), INVALID, "ngroups"), (dict(ngroups=3), INVALID, "multiple"), (dict(nheads=65536), UNSUPPORTED, "nheads"),
    (dict(num_seqs=1 << 19), UNSUPPORTED, "pairs"), (dict(rows=1 << 30), UNSUPPORTED, "2^30"),
    (dict(headdim=128), UNSUPPORTED, "headdim"), (dict(dstate=64), UNSUPPORTED, "dstate"),
    (dict(io_dtype=ssu.SSU_F16), UNSUPPORTED, "io_dtype"), (dict(io_dtype=-7), UNSUPPORTED, "io_dtype"),
    (dict(out_dtype=ssu.SSU_F16), UNSUPPORTED, "out_dtype"), (dict(out_dtype=99), UNSUPPORTED, "out_dtype"),
    (dict(cu_seqlens=None), INVALID, "NULL"), (dict(A=None), INVALID, "NULL"), (dict(D=None), INVALID, "NULL"),
    (dict(dt_bias=None), INVALID, "NULL"), (dict(x=None), INVALID, "NULL"), (dict(B=None), INVALID, "NULL"),
    (dict(C=None), INVALID, "NULL"), (dict(dt=None), INVALID, "NULL"), (dict(out=None), INVALID, "NULL"),
    (dict(x=FAKE + 8), INVALID, "16-byte"), (dict(B=FAKE + 2), INVALID, "16-byte"), (dict(C=FAKE + 4), INVALID, "16-byte"),
    (dict(z=FAKE + 8, z_row_stride=256), INVALID, "16-byte"), (dict(out=FAKE + 8), INVALID, "16-byte"),
    (dict(initial_states=FAKE + 4), INVALID, "16-byte"), (dict(final_states=FAKE + 4), INVALID, "16-byte"),
    (dict(dt=FAKE + 2), INVALID, "4-byte"), (dict(A=FAKE + 1), INVALID, "4-byte"), (dict(D=FAKE + 2), INVALID, "4-byte"),
    (dict(dt_bias=FAKE + 2), INVALID, "4-byte"), (dict(cu_seqlens=FAKE + 2), INVALID, "4-byte"),
    (dict(status=FAKE + 2), INVALID, "4-byte"), (dict(x_row_stride=248), INVALID, "x_row_stride"),
    (dict(x_row_stride=260), INVALID, "x_row_stride"), (dict(B_row_stride=128), INVALID, "B_row_stride"),
    (dict(C_row_stride=264 + 4), INVALID, "C_row_stride"), (dict(z=FAKE), INVALID, "z_row_stride"),
    (dict(x_row_stride=1 << 23), UNSUPPORTED, "2^23"), (dict(workspace=FAKE + 8), INVALID, "workspace"),
    (dict(rows=1 << 20, workspace=None), WORKSPACE, "workspace"), (dict(rows=1 << 20, workspace_bytes=16), WORKSPACE, "workspace")])
def test_prefill_refusals(kw, code, words):
    _refused(prompts.ssu_prefill(_prefill(**kw)), code, words)


def test_prefill_no_op_and_sizes():
    assert prompts.ssu_prefill(_prefill(num_seqs=0, cu_seqlens=None, x=None, A=None)) == ssu.SSU_OK
    assert ssu.ssu_last_error() == ""
    assert ssu.prefill_workspace_size(70, 2, 4) == 0 and ssu.ssu_last_error() == ""  # no sequence is cut
    big = ssu.prefill_workspace_size(1 << 20, 1, 4)
    assert big > 0 and big % 8 == 0
    for bad in ((-1, 1, 4), (1, -1, 4), (1, 1, 0), (1 << 30, 1, 4), (1, 1 << 20, 4)):
        assert ssu.prefill_workspace_size(*bad) == 0 and ssu.ssu_last_error() != "", bad
    # room for every way that the rows may be cut into sequences
    for rows in (0, 1, 513, 4096, 100000):
        for n in (1, 2, 63):
            assert ssu.prefill_workspace_size(rows, n, 8) <= ssu.prefill_workspace_size(rows + 4096, n + 1, 8)


def _cache(**kw):
    return _fill(ssu.SsuCache(), dict(
        num_slots=8, nheads=4, ngroups=2, headdim=64, dstate=128, ring_len=16, state_dtype=ssu.SSU_FP8_E4M3, io_dtype=ssu.SSU_BF16,
        state=FAKE, state_slot_stride=4 * 8192, state_scale=FAKE, scale_slot_stride=4 * 256, x_cache=FAKE,
        x_slot_stride=4 * 16 * 128, B_cache=FAKE, B_slot_stride=2 * 16 * 256, dt_cache=FAKE, dt_slot_stride=4 * 16 * 4,
        ring_start=FAKE), kw)


PACKED = 4 * 8192


@pytest.mark.parametrize("cache,args,code,words", [
    (dict(num_slots=0), (FAKE, PACKED, FAKE, 2, 0), INVALID, "num_slots"),
    (dict(headdim=128), (FAKE, PACKED, FAKE, 2, 0), UNSUPPORTED, "headdim"),
    ({}, (FAKE, PACKED, FAKE, -1, 0), INVALID, "n must"), ({}, (FAKE, PACKED, FAKE, 1 << 20, 0), UNSUPPORTED, "pairs"),
    ({}, (FAKE, PACKED, FAKE, 2, 1), INVALID, "recur_state"), ({}, (None, PACKED, FAKE, 2, 0), INVALID, "NULL"),
    ({}, (FAKE, PACKED, None, 2, 0), INVALID, "NULL"), ({}, (FAKE, PACKED - 4, FAKE, 2, 0), INVALID, "stride"),
    ({}, (FAKE, 0, FAKE, 2, 0), INVALID, "stride"), ({}, (FAKE, PACKED + 2, FAKE, 2, 0), INVALID, "stride"),
    ({}, (FAKE + 8, PACKED, FAKE, 2, 0), INVALID, "16-byte"), ({}, (FAKE, PACKED, FAKE + 2, 2, 0), INVALID, "4-byte")])
def test_read_state_refusals(cache, args, code, words):
    _refused(prompts.ssu_read_state(_cache(**cache), *args), code, words)


def test_read_state_no_op():
    assert prompts.ssu_read_state(_cache(), None, 0, None, 0, 1) == ssu.SSU_OK


def _history(**kw):
    return _fill(ssu.SsuHistory(), dict(num_slots=5, vocab=1000, counts=FAKE, counts_slot_stride=4000, seen=FAKE,
                                        seen_slot_stride=128), kw)


def _count(**kw):
    return _fill(ssu.SsuCount(), dict(batch=3, max_seqlen=4, rows=12, slot_idx=FAKE, tokens=FAKE, num_tokens=FAKE), kw)


BAD_HISTORIES = [
    (dict(num_slots=0), INVALID, "num_slots"), (dict(vocab=0), INVALID, "vocab"), (dict(vocab=(1 << 24) + 1), UNSUPPORTED, "vocab"),
    (dict(counts=None), INVALID, "NULL"), (dict(seen=None), INVALID, "NULL"), (dict(counts=FAKE + 2), INVALID, "4-byte"),
    (dict(seen=FAKE + 1), INVALID, "4-byte"), (dict(status=FAKE + 2), INVALID, "4-byte"),
    (dict(counts_slot_stride=3996), INVALID, "counts"), (dict(counts_slot_stride=4002), INVALID, "counts"),
    (dict(seen_slot_stride=124), INVALID, "seen"), (dict(seen_slot_stride=130), INVALID, "seen")]


@pytest.mark.parametrize("kw,code,words", BAD_HISTORIES)
def test_history_refusals(kw, code, words):
    _refused(sampling.ssu_history_count(_history(**kw), _count()), code, words)
    _refused(sampling.ssu_logits(_history(**kw), _logits()), code, words)


@pytest.mark.parametrize("kw,code,words", [
    (dict(batch=-1), INVALID, "batch"), (dict(batch=(1 << 20) + 1), UNSUPPORTED, "batch"), (dict(rows=-1), INVALID, "rows"),
    (dict(max_seqlen=0), INVALID, "max_seqlen"), (dict(slot_idx=None), INVALID, "NULL"), (dict(tokens=None), INVALID, "NULL"),
    (dict(cu_seqlens=FAKE), INVALID, "exclude"), (dict(rows=11), INVALID, "hold no"), (dict(slot_idx=FAKE + 2), INVALID, "4-byte"),
    (dict(tokens=FAKE + 2), INVALID, "4-byte"), (dict(num_tokens=FAKE + 2), INVALID, "4-byte"),
    (dict(num_tokens=None, cu_seqlens=FAKE + 2), INVALID, "4-byte")])
def test_count_refusals(kw, code, words):
    _refused(sampling.ssu_history_count(_history(), _count(**kw)), code, words)


def test_count_no_op():
    assert sampling.ssu_history_count(_history(), _count(batch=0, slot_idx=None, tokens=None, rows=0)) == ssu.SSU_OK


def _logits(**kw):
    return _fill(ssu.SsuLogits(), dict(
        batch=3, max_seqlen=4, rows=12, vocab=1000, logits_dtype=ssu.SSU_BF16, out_dtype=ssu.SSU_F32, logits=FAKE,
        logits_row_stride=1000, out=FAKE * 2, out_row_stride=1000, slot_idx=FAKE, tokens=FAKE, workspace=FAKE,
        workspace_bytes=1 << 20), kw)


@pytest.mark.parametrize("kw,code,words", [
    (dict(batch=-1), INVALID, "batch"), (dict(max_seqlen=0), INVALID, "max_seqlen"), (dict(max_seqlen=65), UNSUPPORTED, "max_seqlen"),
    (dict(vocab=0), INVALID, "vocab"), (dict(vocab=(1 << 24) + 1), UNSUPPORTED, "vocab"), (dict(batch=16384), UNSUPPORTED, "65535"),
    (dict(batch=16000, vocab=1 << 24), UNSUPPORTED, "2^23"), (dict(vocab=999), INVALID, "history"),
    (dict(logits_dtype=ssu.SSU_FP8_E4M3), UNSUPPORTED, "dtype"), (dict(out_dtype=-1), UNSUPPORTED, "dtype"),
    (dict(rows=-1), INVALID, "rows"), (dict(rows=11), INVALID, "hold no"), (dict(logits=None), INVALID, "NULL"),
    (dict(out=None), INVALID, "NULL"), (dict(slot_idx=None), INVALID, "slot_idx"), (dict(logits=FAKE + 1), INVALID, "aligned"),
    (dict(out=FAKE + 2), INVALID, "aligned"), (dict(logits_row_stride=999), INVALID, "stride"),
    (dict(out_row_stride=999), INVALID, "stride"), (dict(out=FAKE), INVALID, "in place"),
    (dict(out=FAKE, out_dtype=ssu.SSU_BF16, out_row_stride=1008), INVALID, "in place"),
    (dict(cu_seqlens=FAKE + 2), INVALID, "4-byte"), (dict(tokens=FAKE + 2), INVALID, "4-byte"),
    (dict(temperature=FAKE + 2), INVALID, "4-byte"), (dict(mask=FAKE + 2), INVALID, "4-byte"), (dict(status=FAKE + 1), INVALID, "4-byte"),
    (dict(bias_offsets=FAKE + 2), INVALID, "4-byte"), (dict(bias_count=-1), INVALID, "bias_count"),
    (dict(bias_count=1 << 24), INVALID, "bias_count"), (dict(bias_offsets=FAKE, bias_count=2), INVALID, "bias_tokens"),
    (dict(mask=FAKE, mask_row_stride=31), INVALID, "mask_row_stride"), (dict(mask=FAKE, mask_row_stride=-32), INVALID, "mask_row_stride"),
    (dict(workspace=None), WORKSPACE, "workspace"), (dict(workspace_bytes=95), WORKSPACE, "workspace"),
    (dict(workspace=FAKE + 8), INVALID, "workspace")])
def test_logits_refusals(kw, code, words):
    _refused(sampling.ssu_logits(_history(), _logits(**kw)), code, words)


@pytest.mark.parametrize("name", ["repetition", "frequency", "presence"])
def test_logits_penalties_need_a_history(name):
    _refused(sampling.ssu_logits(None, _logits(**{name: FAKE})), INVALID, "history")


def test_logits_no_op_and_sizes():
    assert sampling.ssu_logits(None, _logits(batch=0, logits=None, out=None, workspace=None)) == ssu.SSU_OK
    assert ssu.logits_workspace_size(3, 4, 1000) == 96
    for bad in ((-1, 1, 5), (1, 0, 5), (1, 65, 5), (1, 1, 0), (1, 1, (1 << 24) + 1), (65536, 1, 5)):
        assert ssu.logits_workspace_size(*bad) == 0 and ssu.ssu_last_error() != "", bad


def test_null_descriptors():
    lib = ctypes.CDLL(ssu.LIB_PATH)
    assert lib.ssu_prefill(None, None) == INVALID and lib.ssu_logits(None, None, None) == INVALID
    assert lib.ssu_history_count(None, None, None) == INVALID and lib.ssu_read_state(None, None, 0, None, 0, 0, None) == INVALID
    assert lib.ssu_history_count(ctypes.byref(_history()), None, None) == INVALID


def test_front_end_refuses_host_tensors():
    i32, f32 = torch.zeros(3, dtype=torch.int32), torch.zeros(4)
    x = torch.zeros(8, 4, 64, dtype=torch.bfloat16)
    b = torch.zeros(8, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        ssu.make_prefill(i32, x, b, b, torch.zeros(8, 4), f32, f32, f32, x)
    with pytest.raises(ValueError, match="device tensor"):
        ssu.TokenHistory(2, 64, torch.zeros(2, 64, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        ssu.make_logits(torch.zeros(3, 64), torch.zeros(3, 64), 3, 1)
