"""First calls of the operators' binding from two threads at once, on the CPU:
wherever one thread stands in its look-up of the device functions, another one's
call goes through."""
import sys
import threading

import torch

import quantized_linear_layer_amd as qll


class OnDevice:
    def get_device(self):
        return 0


def test_first_call_interrupted_anywhere(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 64 + dev, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    failed, places = [], set()

    def call():
        try:
            assert qll._device(OnDevice(), "x") == 0 and qll._on(0, None) == 64
        except BaseException as e:
            failed.append(e)

    def interrupted_at(place):
        """A first call that another thread's whole call interrupts before the
        instruction at `place`; None: collects the places."""
        monkeypatch.setattr(qll, "_raw_stream", None)
        monkeypatch.setattr(qll, "_current_device", None)

        def trace(frame, event, arg):
            if frame.f_code is not qll._device.__code__:
                return None
            frame.f_trace_opcodes = True
            if event == "opcode" and place is None:
                places.add(frame.f_lasti)
            elif event == "opcode" and frame.f_lasti == place:
                other = threading.Thread(target=call)
                other.start()
                other.join()
            return trace

        before = sys.gettrace()
        sys.settrace(trace)
        try:
            call()
        finally:
            sys.settrace(before)

    interrupted_at(None)
    assert not failed and len(places) > 10
    for place in sorted(places):
        interrupted_at(place)
        assert not failed, f"before the instruction at {place}: {failed[0]!r}"
