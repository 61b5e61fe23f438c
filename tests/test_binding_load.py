"""Without the built library the binding's calls fail at once, and say why."""
import threading

from linear_attention_chunk_gb300 import binding


def test_a_missing_library_is_an_error_not_a_wait(monkeypatch):
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "LIB_PATH", "/nonexistent/libgla.so")
    monkeypatch.setattr(binding, "_lock", threading.Lock())
    seen = []

    def call():
        try:
            binding.gla_version()
        except binding.GlaError as e:
            seen.append(e)
    for _ in range(2):                                      # the lock is free again after the first
        t = threading.Thread(target=call, daemon=True)
        t.start()
        t.join(5)
        assert not t.is_alive(), "the call waits on the loader's own lock"
    assert len(seen) == 2 and all(e.status == binding.GLA_ERR_CUDA and "is not built" in str(e) for e in seen)


def test_an_error_before_the_first_call_has_the_library_s_name(monkeypatch):
    from linear_attention_chunk_gb300.build import build
    build()
    monkeypatch.setattr(binding, "_lib", None)
    e = binding.GlaError(binding.GLA_ERR_WORKSPACE, "f")
    assert binding.gla_status_string(binding.GLA_ERR_WORKSPACE) in str(e)
