"""A grouped call asks for its workspace on the device of its tensors, whichever
is current (CPU only: the device switch and the query are recorded)."""
import pytest
import torch

from bit_quantized_lora_blockwise_b200 import binding


@pytest.mark.parametrize("offsets", [True, False])
def test_workspace_is_sized_on_the_tensors_device(monkeypatch, offsets):
    E, T, N, K, r = (2, 8, 64, 64, 8) if offsets else (1, 8, 64, 64, 8)
    current = ["another"]

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, current[0] = current[0], self.device

        def __exit__(self, *exc):
            current[0] = self.before

    asked = []

    def query(*shape):
        asked.append((shape, current[0]))
        return 4096

    monkeypatch.setattr(binding, "_on", On)
    monkeypatch.setattr(binding, "grouped_workspace_bytes", query)
    monkeypatch.setattr(binding, "_req", lambda t, *a: t)
    monkeypatch.setattr(binding, "_need", lambda t, *a: t)
    bf = torch.bfloat16
    X, A, B = torch.zeros(T, K, dtype=bf), torch.zeros(E, K, r, dtype=bf), torch.zeros(E, r, N, dtype=bf)
    off = torch.zeros(E + 1, dtype=torch.int32) if offsets else None
    *_, workspace = binding._grouped_checks(None, None, None, X, off, A, B, N, K, None, None,
                                            binding._expert_adapters(A, B, N, K))
    assert asked == [((E, T, N, K, r, False), X.device)] and current == ["another"]
    assert workspace.device == X.device and workspace.numel() == 4096
