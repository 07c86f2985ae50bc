"""Shapes of grouped products, each with the kernel that the library's rule takes for it on a B200's
148 SMs: "simt" (fp32) and "warp" (bf16 that TMA cannot take) with the tiles' side and the elements
a load, "tma" with the rows per tile, or for weight gradients with the parts of the rows.

Contractions are long enough for several steps, and for several pieces of the sums that are added up
apart (256 values fp32, 480 the warp kernel's weight gradients, 384 the tensor cores')."""

TAIL = 7   # rows of the buffers behind the last expert's

# (op, dtype, counts, n, k, kernel)
CASES = [
    ("mm", "fp32", [2400, 2301, 0, 2377, 1999, 300], 1024, 1028, "simt 128 4"),
    ("mm", "fp32", [2400, 2301, 0, 2377, 1999, 300], 1001, 1003, "simt 128 1"),
    ("dgrad", "fp32", [2400, 2301, 0, 2377, 1999, 300], 1028, 1024, "simt 128 4"),
    ("dgrad", "fp32", [2400, 2301, 0, 2377, 1999, 300], 1003, 1001, "simt 128 1"),
    ("wgrad", "fp32", [2400, 2301, 0, 2377, 1999, 300], 1024, 1028, "simt 128 4"),
    ("wgrad", "fp32", [2400, 2301, 0, 2377, 1999, 300], 1001, 1003, "simt 128 1"),
    ("mm", "fp32", [700, 301, 0, 499], 1000, 520, "simt 64 4"),
    ("mm", "fp32", [700, 301, 0, 499], 1001, 523, "simt 64 1"),
    ("dgrad", "fp32", [700, 301, 0, 499], 520, 1000, "simt 64 4"),
    ("dgrad", "fp32", [700, 301, 0, 499], 523, 1001, "simt 64 1"),
    ("wgrad", "fp32", [700, 301, 0, 499], 512, 1000, "simt 64 4"),
    ("wgrad", "fp32", [700, 301, 0, 499], 511, 1001, "simt 64 1"),
    ("mm", "fp32", [70, 301, 0, 49], 130, 1025, "simt 32 1"),
    ("mm", "fp32", [70, 301, 0, 49], 128, 1024, "simt 32 1"),
    ("dgrad", "fp32", [70, 301, 0, 49], 1025, 130, "simt 32 1"),
    ("wgrad", "fp32", [700, 301, 0, 499], 66, 131, "simt 32 1"),
    ("mm", "bf16", [700, 301, 0, 499, 650], 1001, 515, "warp 128"),
    ("dgrad", "bf16", [700, 301, 0, 499, 650], 515, 1001, "warp 128"),
    ("wgrad", "bf16", [700, 301, 0, 499, 650], 1001, 515, "warp 128"),
    ("mm", "bf16", [700, 301, 0, 499, 650], 301, 1015, "warp 64"),
    ("dgrad", "bf16", [700, 301, 0, 499, 650], 1015, 301, "warp 64"),
    ("wgrad", "bf16", [700, 301, 0, 499, 650], 301, 130, "warp 64"),
    ("wgrad", "bf16", [5001, 0, 3000], 130, 131, "warp 64 parts 5"),
    ("wgrad", "fp32", [5001, 0, 3000], 130, 131, "simt 32 1 parts 5"),
    ("mm", "bf16", [30, 51, 0, 35], 520, 1032, "tma 64"),
    ("mm", "bf16", [700, 301, 0, 499], 520, 1032, "tma 256"),
    ("dgrad", "bf16", [30, 51, 0, 35], 1032, 520, "tma 64"),
    ("dgrad", "bf16", [700, 301, 0, 499], 1032, 520, "tma 256"),
    ("wgrad", "bf16", [1700, 301, 0, 499], 520, 264, "tma"),
    ("wgrad", "bf16", [5001, 0, 3000], 136, 264, "tma parts 2"),
    ("wgrad", "bf16", [20001, 3, 0, 1], 64, 136, "tma parts 4"),
    ("wgrad", "bf16", [20001, 3, 0, 1], 33, 35, "warp 64 parts 9"),
    ("wgrad", "fp32", [20001, 3, 0, 1], 64, 40, "simt 32 1 parts 9"),
    ("wgrad", "fp32", [20001, 3, 0, 1], 33, 35, "simt 32 1 parts 9"),
]
