"""The binding of the hybrid layers' calls, without a GPU: what a call does with the status that it gets."""

import pytest
import torch

bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
OK, INVALID_ARG, UNSUPPORTED, CUDA = 0, 1, 13, 14


class _Library:
    """Answers each call with the next of its statuses (the last one for ever) and counts them."""

    def __init__(self, *statuses):
        self.statuses, self.calls = list(statuses), 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return self.statuses[min(self.calls, len(self.statuses)) - 1]
        return call


def _calls(bfp8):
    slots, off = torch.zeros(1, dtype=i32), torch.tensor([0, 4], dtype=i32)
    x, heads = torch.zeros(4, 64, dtype=bf16), torch.zeros(4, 2, 128, dtype=bf16)
    ab, gates = torch.zeros(4, 2, dtype=bf16), torch.zeros(2)
    return {
        "bfp8_causal_conv": lambda: bfp8.bfp8_causal_conv(x, torch.zeros(64, 4, dtype=bf16), torch.empty_like(x), off,
                                                          torch.zeros(2, 3, 64, dtype=bf16), slots, slots),
        "bfp8_delta_rule": lambda: bfp8.bfp8_delta_rule(heads, heads, heads, ab, ab, gates, gates, torch.zeros(2, 2, 128, 128), slots,
                                                        slots, off, torch.empty_like(heads), 4),
        "bfp8_gated_norm": lambda: bfp8.bfp8_gated_norm(heads, heads, torch.zeros(128), torch.empty_like(heads)),
        "bfp8_rotary": lambda: bfp8.bfp8_rotary(heads, heads, torch.zeros(4, dtype=i32), torch.zeros(32)),
    }


@pytest.mark.parametrize("name", ["bfp8_causal_conv", "bfp8_delta_rule", "bfp8_gated_norm", "bfp8_rotary"])
@pytest.mark.parametrize("statuses,made", [((OK,), 1), ((CUDA, OK), 1), ((INVALID_ARG, OK), 2), ((UNSUPPORTED, UNSUPPORTED), 2),
                                           ((INVALID_ARG, CUDA), 2)], ids=str)
def test_a_call_is_made_again_only_where_it_was_refused(bfp8, monkeypatch, name, statuses, made):
    """A refusal has done nothing, and the helpers look for its reason; a CUDA error may come after a launch that moves the
    states, so it is raised and the call not repeated."""
    lib = _Library(*statuses)
    call = _calls(bfp8)[name]
    monkeypatch.setattr(bfp8, "_lib", lib)
    monkeypatch.setattr(bfp8, "_device", lambda: -1)              # the host's tensors stand for the device's
    monkeypatch.setattr(bfp8, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(bfp8, "bfp8_status_string", lambda status: bfp8.STATUS_NAMES[status])
    last = statuses[made - 1]
    if last == OK:
        call()
    else:
        with pytest.raises(bfp8.Bfp8Error, match=bfp8.STATUS_NAMES[last]):
            call()
    assert lib.calls == made
