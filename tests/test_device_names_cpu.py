"""A device given without an index is the current one, as in torch (no GPU:
the library is replaced by one that records the device and refuses)."""
import pytest

torch = pytest.importorskip("torch")

import entropy_bound_canvas_b200 as E


class Recorder:
    """Stands in for the C library: notes the device a handle is asked for."""

    def __init__(self):
        self.device = None

    def eb_config_default(self, *args):
        pass

    def eb_sampler_init(self, out, cfg, device):
        self.device = device
        return 2

    def eb_scorer_init(self, out, max_rows, device):
        self.device = device
        return 2

    def eb_strerror(self, code):
        return b""


@pytest.mark.parametrize("given,want", [
    (None, 3), ("cuda", 3), ("cuda:0", 0), ("cuda:1", 1), (torch.device("cuda"), 3),
    (torch.device("cuda", 2), 2), (0, 0), (1, 1)])
@pytest.mark.parametrize("make", [lambda d: E.EBScorer(16, device=d),
                                  lambda d: E.EBSampler(1, 16, 64, device=d)],
                         ids=["scorer", "sampler"])
def test_the_device_a_handle_is_made_on(monkeypatch, make, given, want):
    lib = Recorder()
    monkeypatch.setattr(E, "_lib", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    with pytest.raises(E.EBError):
        make(given)
    assert lib.device == want
