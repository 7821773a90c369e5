"""ZeroConfig built by position: fields keep their places, new ones come last."""
from dataclasses import fields

from zero_sharded_mixed_gb300.config import ZeroConfig


def test_places():
    names = [f.name for f in fields(ZeroConfig)]
    assert names[:15] == ["stage", "reduce_bucket_size", "gradient_accumulation_steps", "gradient_clipping", "lr", "betas", "eps",
                          "weight_decay", "zero_quantized_weights", "zero_quantized_gradients", "overlap_comm",
                          "stage3_gather_16bit_weights_on_model_save", "quant_block", "scheduler", "ignored"]
    assert names[15:] == ["optimizer", "momentum", "nesterov", "ns_steps"]


def test_by_position():
    cfg = ZeroConfig(3, 1000, 1, 0.0, 1e-3, (0.9, 0.95), 1e-8, 0.1, True, False, True)
    assert cfg.zero_quantized_weights and cfg.overlap_comm and not cfg.zero_quantized_gradients
    assert cfg.optimizer == "adamw"
