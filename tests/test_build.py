"""When the compiled calls are built again (no GPU)."""
from mtp_speculative_decoding_qmv_gb300 import build as b


def test_the_extension_is_stale_for_another_torch(tmp_path, monkeypatch):
    b.build()
    assert not b.checks_stale()
    other = tmp_path / "for"
    monkeypatch.setattr(b, "CHECKS_FOR", other)
    assert b.checks_stale()  # nothing says what it was compiled for
    other.write_text(b.interpreter())
    assert not b.checks_stale()
    import torch

    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert b.checks_stale()
    calls = []
    monkeypatch.setattr(b, "build_checks", lambda: calls.append(1))
    b.build()
    assert calls == [1]
