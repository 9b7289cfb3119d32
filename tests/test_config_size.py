"""CPU: the configuration's size, by which a client knows that the library reads the dfl_config it was built with."""
import ctypes

import pytest


def test_sizes_agree():
    from dflash_speculative_decode_gb300 import _abi
    assert _abi.lib().dfl_config_bytes() == ctypes.sizeof(_abi.dfl_config)


def test_the_binding_refuses_a_library_with_another_configuration(monkeypatch):
    """As a binding of before the last field would find it: nothing is passed to a library that reads more than it gets."""
    from dflash_speculative_decode_gb300 import _abi

    class Before(ctypes.Structure):
        _fields_ = _abi.dfl_config._fields_[:-1]
    assert ctypes.sizeof(Before) < ctypes.sizeof(_abi.dfl_config)
    monkeypatch.setattr(_abi, "_lib", None)
    monkeypatch.setattr(_abi, "dfl_config", Before)
    with pytest.raises(RuntimeError, match="another build"):
        _abi.lib()
