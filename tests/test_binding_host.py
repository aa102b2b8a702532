"""What the binding promises about host threads, without a GPU."""

import ctypes

import quantized_linear_layers_awq_amd as tf


def test_calls_hold_the_interpreter_lock():
    """The linears and the attention calls share one workspace per stream, and
    some of each launch two kernels that hand over partial results in it.  Only
    a call that keeps the interpreter lock from its first launch to its last
    keeps another thread's launches on the same stream out."""
    assert isinstance(tf.load_library(), ctypes.PyDLL)
