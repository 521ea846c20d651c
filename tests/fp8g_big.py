"""Sizes of FP8 with group scales whose operands or results take more than 2^32 bytes, and the kernel that each takes."""
GEMM = [(5_000_001, 1000, 1024, "bf16", "LARGE"), (5_000_001, 1000, 1024, "f32", "LARGE"),
        (9_000_001, 128, 512, "bf16", "SMALL"), (9_000_001, 128, 512, "f32", "SMALL")]
FWD = [(40_000_077, 128, 8, "FEW"), (20_000_005, 1024, 64, "SMALL"), (9_000_005, 512, 512, "LARGE")]
BWD = [(70_000_009, 128, 8, "FEW"), (40_000_005, 128, 128, "GROUP"), (5_000_003, 512, 512, "LARGE")]
