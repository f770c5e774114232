"""The smoke check runs with the library's kernels alone: CUDA's linear algebra,
which torch loads from a library of its own at the first such call, is not used."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_smoke_takes_its_singular_values_on_the_cpu(monkeypatch, capsys):
    import __graft_entry__ as entry
    entry.build()
    svdvals, seen = torch.linalg.svdvals, []

    def on_cpu(a, **kw):
        seen.append(a.device.type)
        assert a.device.type == "cpu"
        return svdvals(a, **kw)

    monkeypatch.setattr(torch.linalg, "svdvals", on_cpu)
    entry.smoke()
    assert seen == ["cpu"]
    assert "smoke ok: shared expert" in capsys.readouterr().out
