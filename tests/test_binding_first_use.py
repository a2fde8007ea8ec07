"""The binding's first use from two threads at once."""

import importlib.util
import os
import sys
import threading

import torch

import sparse_dense_gemm_amd as sdg


def fresh():
    """The binding as a module of its own that nothing has used yet."""
    path = os.path.join(os.path.dirname(sdg.__file__), "__init__.py")
    spec = importlib.util.spec_from_file_location("binding_first_use", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_a_second_thread_at_any_line_of_the_first_use():
    lines, wrong = [], []
    x = torch.zeros(1)
    for stop in range(1, 40):
        m = fresh()
        seen = 0

        def other():
            try:
                if m.dtype_of(x) != m.DT_F32 or m._torch() is not torch:
                    wrong.append((stop, "value"))
            except Exception as e:
                wrong.append((stop, repr(e)))

        def trace(frame, event, arg):
            nonlocal seen
            if frame.f_code.co_filename != m.__file__:
                return None
            if event == "line":
                seen += 1
                if seen == stop:  # the first thread stands still at this line
                    t = threading.Thread(target=other)
                    t.start()
                    t.join()
            return trace

        old = sys.gettrace()
        sys.settrace(trace)
        try:
            first = m.dtype_of(x)
        finally:
            sys.settrace(old)
        assert first == m.DT_F32
        lines.append(seen)
        if seen < stop:
            break
    assert len(lines) > 5 and lines[-1] < len(lines)  # every line of the first use was tried
    assert not wrong
