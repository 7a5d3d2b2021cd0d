"""The LM head's layers where no GPU is needed."""
import contextlib
import threading
import time

import torch

import qlora_linear_b200 as q


def test_capture_id_refuses_no_place_for_it():
    assert q.lib().lora_stream_capture_id(None, None) == q.LORA_ERR_INVALID_ARG


def test_status_while_another_thread_makes_its_first_call_on_a_stream(monkeypatch):
    """status() goes over the streams' workspaces while another thread's call adds one."""
    layer = q.LoraTokenLogProbs(q.LoraWeight.bf16(torch.zeros((64, 32), dtype=torch.bfloat16)))
    ws = torch.zeros(256, dtype=torch.uint8)
    layer._ws = {(0, 1): ws, (0, 2): ws}
    threads = []

    def call(stream):  # as _run and _workspace
        with layer._lock:
            layer._ws[(0, stream)] = ws

    def read(workspace, stream):
        threads.append(threading.Thread(target=call, args=(10 + len(threads),)))
        threads[-1].start()
        time.sleep(0.05)
        return q.LORA_ERR_DEVICE_TIMEOUT if stream == 2 else q.LORA_OK

    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(q.head._b, "lora_device_status", read)
    assert layer.status() == q.LORA_ERR_DEVICE_TIMEOUT
    for t in threads:
        t.join(timeout=10)
    assert len(layer._ws) == 4
