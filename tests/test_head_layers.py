"""The LM head's layers where no GPU is needed."""
import qlora_linear_b200 as q


def test_capture_id_refuses_no_place_for_it():
    assert q.lib().lora_stream_capture_id(None, None) == q.LORA_ERR_INVALID_ARG
