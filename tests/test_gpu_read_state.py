"""ssu_read_state on the GPU: every checkpoint's values exactly (one rounding
to fp32 where there is a scale), slots that nobody named left alone."""
import numpy as np
import pytest
import torch

import synth
from synth import device as sd

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import speculative_replay_state_amd as ssu
    from oracle import ssu_oracle as O
    from tests import gpu_harness as GH

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def spec_of(state, H=3, slots=6, **kw):
    return synth.CacheSpec(num_slots=slots, nheads=H, ngroups=1, state_dtype=state, separate=kw.pop("separate", state == "nvfp4"), **kw)


@pytest.mark.parametrize("state,separate", [("f32", False), ("bf16", False), ("f16", False), ("fp8", False), ("fp8", True), ("nvfp4", True)])
@pytest.mark.parametrize("H", [1, 3, 16])
def test_values(state, separate, H):
    spec = spec_of(state, H, separate=separate)
    cache = synth.make_cache(spec, 11)
    t = sd.upload_cache(cache, DEV)
    dc = GH.device_cache(spec, t)
    ids = [4, 0, 2, -1, 5, 6, 2]   # padding, out of range, and one of them twice
    wide = torch.full((len(ids), H * 8192 + 8), -7.0, device=DEV)
    states = wide[:, :H * 8192].unflatten(1, (H, 64, 128))  # entries with a gap between them
    for recur in ([False, True] if separate else [False]):
        wide.fill_(-7.0)
        ssu.read_state(dc, states, torch.tensor(ids, dtype=torch.int32, device=DEV), recur=recur)
        got = wide.cpu().numpy()
        assert (got[:, H * 8192:] == -7).all()
        for j, slot in enumerate(ids):
            if slot < 1 or slot >= spec.num_slots:
                assert (got[j] == -7).all()
                continue
            want = (O.decode_recur(cache, slot) if recur else O.decode_state(cache, slot)).astype(np.float32)
            assert np.array_equal(got[j, :H * 8192], want.reshape(-1)), (j, slot)
    after = sd.download_cache(spec, t)
    for f in ("state", "scale", "x_cache", "B_cache", "dt_cache", "ring_start", "recur", "gscale"):
        a, b = getattr(after, f), getattr(cache, f)
        assert (a is None and b is None) or np.array_equal(a, b), f


@pytest.mark.parametrize("state", ["f32", "bf16", "f16", "fp8", "nvfp4"])
def test_init_of_what_was_read_gives_the_checkpoint_back(state):
    spec = spec_of(state, 2)
    cache = synth.make_cache(spec, 12)
    t = sd.upload_cache(cache, DEV)
    dc = GH.device_cache(spec, t)
    ids = torch.tensor([1, 3], dtype=torch.int32, device=DEV)
    states = torch.empty(2, 2, 64, 128, device=DEV)
    ssu.read_state(dc, states, ids)
    again = torch.empty_like(states)
    ssu.init_state(dc, states, ids)
    ssu.read_state(dc, again, ids)
    if state in ("f32", "bf16", "f16"):
        assert torch.equal(again, states)
    else:  # a scale that is taken from the values again moves them by no more than the type's own step
        worst = ((again - states).abs().amax(-1) / states.abs().amax(-1)).max()
        assert float(worst) <= (2.0 ** -4 if state == "fp8" else 2.0 ** -1)


def test_infinities_and_nan_come_out():
    spec = spec_of("bf16", 1)
    cache = synth.make_cache(spec, 13)
    t = sd.upload_cache(cache, DEV)
    v = t["state"][2].view(torch.bfloat16)
    v[5], v[6], v[7] = float("inf"), float("-inf"), float("nan")
    states = torch.empty(1, 1, 64, 128, device=DEV)
    ssu.read_state(GH.device_cache(spec, t), states, torch.tensor([2], dtype=torch.int32, device=DEV))
    assert int(torch.isnan(states).sum()) == 1 and int((states == float("inf")).sum()) == 1 and int((states == float("-inf")).sum()) == 1


def test_slot_pages_past_4_GiB():
    H, slots = 16, 3
    page = (1 << 31) + 64
    state = torch.empty(slots * page, dtype=torch.uint8, device=DEV).as_strided((slots, H * 8192 * 2), (page, 1))
    want = torch.randn(H, 64, 128, device=DEV).bfloat16().float()
    small = lambda n: torch.zeros(slots, n, dtype=torch.uint8, device=DEV)  # noqa: E731
    dc = ssu.DeviceCache(slots, H, 1, 16, "bf16", state, None, small(H * 16 * 128), small(16 * 256), small(H * 16 * 4),
                         torch.zeros(slots, dtype=torch.int32, device=DEV))
    ids = torch.tensor([2], dtype=torch.int32, device=DEV)
    ssu.init_state(dc, want[None], ids)
    got = torch.empty(1, H, 64, 128, device=DEV)
    ssu.read_state(dc, got, ids)
    assert torch.equal(got[0], want)


def test_front_end_refusals():
    spec = spec_of("bf16", 2)
    dc = GH.device_cache(spec, sd.upload_cache(synth.make_cache(spec, 14), DEV))
    ids = torch.tensor([1, 2], dtype=torch.int32, device=DEV)
    good = torch.empty(2, 2, 64, 128, device=DEV)
    for states, idx in ((good.bfloat16(), ids), (good[:1], ids), (good.cpu(), ids), (good, ids.long()), (good, ids.cpu()),
                        (torch.empty(2, 2, 128, 64, device=DEV).transpose(2, 3), ids), (good[:1].expand(2, -1, -1, -1), ids)):
        with pytest.raises(ValueError):
            ssu.read_state(dc, states, idx)
    with pytest.raises(ssu.SsuError) as e:
        ssu.read_state(dc, good, ids, recur=True)
    assert e.value.code == ssu.SSU_ERR_INVALID
    ssu.read_state(dc, good[:0], ids[:0])  # none
