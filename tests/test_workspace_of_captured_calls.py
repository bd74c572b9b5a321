"""Whether a call is under graph capture, as its default workspace goes by: the
answer is that of the call's own stream, on whatever device (torch's calls
stand-ins, no GPU needed)."""
import contextlib

import pytest
import torch

import speculative_sampling_verification_vocab_amd as sv


class Streams:
    """Two devices' current streams, of which some are under capture."""

    def __init__(self, current, captured):
        self.at = [("stream", i) for i in range(2)]
        self.device, self.captured = current, captured

    @contextlib.contextmanager
    def stream(self, s):
        kept = self.device, list(self.at)
        self.device, self.at[s[1]] = s[1], s
        yield
        self.device, self.at = kept


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("captured", [0, 1, None])
@pytest.mark.parametrize("own", [0, 1])
@pytest.mark.parametrize("explicit", [False, True])
def test_the_calls_own_stream_decides(monkeypatch, current, captured, own, explicit):
    side = ("side", own)
    want = side if explicit else ("stream", own)
    st = Streams(current, side if explicit and captured == own else ("stream", captured))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: st.device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: st.at[torch.device(d).index])
    monkeypatch.setattr(torch.cuda, "stream", st.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: st.at[st.device] == st.captured)
    assert sv._capturing(torch.device("cuda", own), side if explicit else None) == (st.captured == want)
    assert st.device == current
