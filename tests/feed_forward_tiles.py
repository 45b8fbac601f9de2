"""Sizes that reach every kernel the feed-forward products have, each with a remainder somewhere.

A line: operator (linear, gated: forward; lb: linear's gradients behind an activation, l0: without one; gb: gated's),
type, m, n, k, whether rows are 16-byte aligned, and how the library says it runs that product on a whole MI355X: forward,
or the gradient named first.  A change of the planner's prices fails the host test until other sizes reach the same
kernels again.
"""
import convolution_forward_conv2d_amd as mic

F32, BF16, E4M3 = mic.MIC_DTYPE_F32, mic.MIC_DTYPE_BF16, mic.MIC_DTYPE_F8_E4M3

LINES = """
gated bf16 199 8377 65 odd any 128x128
gated bf16 69 2755 1035 odd any 128x128 split 4
gated bf16 41 67 65 odd any 64x64
gated bf16 41 64 1032 aligned any 64x64 split 4
gated bf16 259 65 72 aligned fast 128x128
gated bf16 2741 97 1035 odd fast 128x128 pack
gated bf16 267 64 1032 aligned fast 128x128 split 4
gated bf16 885 417 2049 odd fast 128x128 split 3 pack
gated bf16 261 8496 72 aligned fast 128x256
gated bf16 41 4192 1032 aligned fast 128x256 split 4
gated bf16 533 8184 72 aligned fast 192x256
gated bf16 2049 2739 65 odd fast 192x256 pack
gated bf16 41 8472 2056 aligned fast 192x256 split 3
gated bf16 43 65 520 aligned fast 256x128
gated bf16 1161 1707 1035 odd fast 256x128 pack
gated bf16 65 2104 1032 aligned fast 256x128 split 4
gated bf16 389 8432 72 aligned fast 256x192
gated bf16 5051 803 65 odd fast 256x192 pack
gated bf16 599 8345 72 aligned fast 256x256
gated bf16 2307 2587 129 odd fast 256x256 pack
gated e4m3 199 8377 65 odd any 128x128
gated e4m3 69 2801 2049 odd any 128x128 split 4
gated e4m3 41 67 65 odd any 64x64
gated e4m3 41 71 1035 odd any 64x64 split 2
gated e4m3 41 64 272 aligned fast 128x128
gated e4m3 41 65 2064 aligned fast 128x128 split 4
gated e4m3 533 8184 80 aligned fast 192x256
gated e4m3 4399 2815 65 odd fast 192x256 pack
gated e4m3 389 8433 80 aligned fast 256x192
gated e4m3 6547 2501 129 odd fast 256x192 pack
gated e4m3 599 8344 80 aligned fast 256x256
gated e4m3 3493 8267 65 odd fast 256x256 pack
gated e4m3-fast 199 8377 65 odd any 128x128
gated e4m3-fast 69 2801 2049 odd any 128x128 split 4
gated e4m3-fast 41 67 65 odd any 64x64
gated e4m3-fast 41 71 1035 odd any 64x64 split 2
gated e4m3-fast 267 64 144 aligned fast 128x128
gated e4m3-fast 259 65 1035 odd fast 128x128 pack
gated e4m3-fast 259 64 2064 aligned fast 128x128 split 4
gated e4m3-fast 261 8497 80 aligned fast 128x256
gated e4m3-fast 41 4193 2064 aligned fast 128x256 split 4
gated e4m3-fast 533 8184 80 aligned fast 192x256
gated e4m3-fast 517 8557 129 odd fast 192x256 pack
gated e4m3-fast 41 64 272 aligned fast 256x128
gated e4m3-fast 1161 1707 1035 odd fast 256x128 pack
gated e4m3-fast 41 65 2064 aligned fast 256x128 split 4
gated e4m3-fast 389 8432 80 aligned fast 256x192
gated e4m3-fast 579 6653 129 odd fast 256x192 pack
gated e4m3-fast 599 8345 80 aligned fast 256x256
gated e4m3-fast 1025 5409 129 odd fast 256x256 pack
gated f32 199 8377 65 odd any 128x128
gated f32 41 2185 2049 odd any 128x128 split 13
gated f32 129 8867 65 odd any 64x64
gated f32 65 8944 72 aligned fast 128x128
gated f32 65 8201 65 odd fast 128x128 pack
gated f32 65 2736 1032 aligned fast 128x128 split 5
gated f32 69 2755 1035 odd fast 128x128 split 5 pack
gated f32 41 64 72 aligned fast 128x64
gated f32 41 67 65 odd fast 128x64 pack
gated f32 43 64 520 aligned fast 128x64 split 4
gated f32 41 67 333 odd fast 128x64 split 2 pack
gated f32 41 8225 72 aligned fast 64x128
gated f32 41 8363 65 odd fast 64x128 pack
gated f32 41 2072 520 aligned fast 64x128 split 4
gated f32 41 1205 1035 odd fast 64x128 split 7 pack
gb bf16 41 201 8681 odd dw any 128x128
gb bf16 1241 2049 65 odd dw any 128x128 split 5
gb bf16 41 65 67 odd dw any 64x64
gb bf16 463 65 67 odd dw any 64x64 split 2
gb bf16 71 136 64 aligned dw fast 128x128
gb bf16 521 129 67 odd dw fast 128x128 pack b
gb bf16 843 136 64 aligned dw fast 128x128 split 3
gb bf16 1347 2049 69 odd dw fast 128x128 split 4 pack b
gb bf16 41 520 6616 aligned dw fast 128x256
gb bf16 333 2485 3261 odd dw fast 128x256 pack b
gb bf16 72 5568 984 aligned dw fast 192x256
gb bf16 65 5463 973 odd dw fast 192x256 pack b
gb bf16 6959 136 5472 aligned dw fast 192x256 split 5
gb bf16 520 48 64 aligned dw fast 256x128
gb bf16 535 2049 999 odd dw fast 256x128 pack b
gb bf16 681 72 64 aligned dw fast 256x128 split 2
gb bf16 5565 2049 407 odd dw fast 256x128 split 3 pack b
gb bf16 43 520 7216 aligned dw fast 256x192
gb bf16 65 451 8325 odd dw fast 256x192 pack b
gb bf16 43 1032 5448 aligned dw fast 256x256
gb bf16 41 2049 5979 odd dw fast 256x256 pack b
gb bf16 2049 41 2031 odd dx any 128x128
gb bf16 65 449 5607 odd dx any 128x128 split 4
gb bf16 41 65 67 odd dx any 64x64
gb bf16 47 201 65 odd dx any 64x64 split 2
gb bf16 264 48 64 aligned dx fast 128x128
gb bf16 1035 259 65 odd dx fast 128x128 pack b
gb bf16 264 392 64 aligned dx fast 128x128 split 3
gb bf16 1663 2049 65 odd dx fast 128x128 split 11 pack b
gb bf16 1032 48 6608 aligned dx fast 128x256
gb bf16 6419 333 1269 odd dx fast 128x256 pack b
gb bf16 41 2056 2352 aligned dx fast 128x256 split 14
gb bf16 2056 48 5544 aligned dx fast 192x256
gb bf16 2049 41 5447 odd dx fast 192x256 pack b
gb bf16 136 3656 5448 aligned dx fast 192x256 split 9
gb bf16 41 136 72 aligned dx fast 256x128
gb bf16 2049 259 2107 odd dx fast 256x128 pack b
gb bf16 72 5256 64 aligned dx fast 256x128 split 28
gb bf16 1035 3933 1165 odd dx fast 256x128 split 5 pack b
gb bf16 1032 48 7232 aligned dx fast 256x192
gb bf16 2049 43 3969 odd dx fast 256x192 pack b
gb bf16 136 2168 8264 aligned dx fast 256x192 split 5
gb bf16 2056 48 5952 aligned dx fast 256x256
gb bf16 1541 65 7239 odd dx fast 256x256 pack b
gb f32 41 201 8681 odd dw any 128x128
gb f32 2049 41 4219 odd dw any 128x128 split 13
gb f32 41 65 8363 odd dw any 64x64
gb f32 41 72 8224 aligned dw fast 128x128
gb f32 65 65 8201 odd dw fast 128x128 pack b
gb f32 1415 72 2712 aligned dw fast 128x128 split 5
gb f32 1035 2839 65 odd dw fast 128x128 split 5 pack b
gb f32 41 72 64 aligned dw fast 128x64
gb f32 41 65 67 odd dw fast 128x64 pack b
gb f32 293 72 64 aligned dw fast 128x64 split 2
gb f32 333 41 67 odd dw fast 128x64 split 2 pack b
gb f32 1035 41 6105 odd dx any 128x128
gb f32 65 295 8361 odd dx any 128x128 split 5
gb f32 2049 61 1941 odd dx any 64x64
gb f32 200 48 8224 aligned dx fast 128x128
gb f32 201 41 8681 odd dx fast 128x128 pack b
gb f32 65 520 5528 aligned dx fast 128x128 split 5
gb f32 65 449 5607 odd dx fast 128x128 split 5 pack b
gb f32 41 72 64 aligned dx fast 128x64
gb f32 41 65 67 odd dx fast 128x64 pack b
gb f32 41 136 72 aligned dx fast 128x64 split 2
gb f32 41 129 65 odd dx fast 128x64 split 2 pack b
gb f32 136 48 8248 aligned dx fast 64x128
gb f32 129 41 8319 odd dx fast 64x128 pack b
gb f32 41 264 4112 aligned dx fast 64x128 split 4
gb f32 41 333 3481 odd dx fast 64x128 split 5 pack b
l0 bf16 513 333 65 odd dw fast 128x128 pack a pack b
l0 bf16 1929 1035 711 odd dw fast 128x128 split 3 pack a pack b
l0 bf16 65 1555 6917 odd dw fast 192x256 pack a pack b
l0 bf16 877 2049 2033 odd dw fast 256x128 pack a pack b
l0 bf16 65 1695 4801 odd dw fast 256x192 pack a pack b
l0 bf16 129 4949 2325 odd dw fast 256x256 pack a pack b
l0 bf16 333 513 65 odd dx fast 128x128 pack a pack b
l0 bf16 1035 1929 711 odd dx fast 128x128 split 3 pack a pack b
l0 bf16 2669 65 4441 odd dx fast 192x256 pack a pack b
l0 bf16 2049 877 2033 odd dx fast 256x128 pack a pack b
l0 bf16 1695 65 4801 odd dx fast 256x192 pack a pack b
l0 bf16 4949 129 2325 odd dx fast 256x256 pack a pack b
l0 f32 65 199 8377 odd dw fast 128x128 pack a pack b
l0 f32 771 65 5513 odd dw fast 128x128 split 5 pack a pack b
l0 f32 41 65 67 odd dw fast 128x64 pack a pack b
l0 f32 333 41 67 odd dw fast 128x64 split 2 pack a pack b
l0 f32 41 129 8319 odd dw fast 64x128 pack a pack b
l0 f32 1035 43 2315 odd dw fast 64x128 split 7 pack a pack b
l0 f32 199 65 8377 odd dx fast 128x128 pack a pack b
l0 f32 65 771 5513 odd dx fast 128x128 split 5 pack a pack b
l0 f32 41 65 67 odd dx fast 128x64 pack a pack b
l0 f32 41 333 67 odd dx fast 128x64 split 2 pack a pack b
l0 f32 129 41 8319 odd dx fast 64x128 pack a pack b
l0 f32 43 1035 2315 odd dx fast 64x128 split 7 pack a pack b
lb bf16 41 2049 2031 odd dw any 128x128
lb bf16 925 65 5683 odd dw any 128x128 split 3
lb bf16 41 65 67 odd dw any 64x64
lb bf16 463 65 67 odd dw any 64x64 split 2
lb bf16 71 264 64 aligned dw fast 128x128
lb bf16 513 333 65 odd dw fast 128x128 pack b
lb bf16 833 264 64 aligned dw fast 128x128 split 3
lb bf16 2049 3351 65 odd dw fast 128x128 split 7 pack b
lb bf16 43 1032 6608 aligned dw fast 128x256
lb bf16 333 4911 3233 odd dw fast 128x256 pack b
lb bf16 2056 48 4792 aligned dw fast 128x256 split 7
lb bf16 41 2056 5544 aligned dw fast 192x256
lb bf16 65 1323 8079 odd dw fast 192x256 pack b
lb bf16 4391 136 8224 aligned dw fast 192x256 split 6
lb bf16 520 48 64 aligned dw fast 256x128
lb bf16 605 2049 1993 odd dw fast 256x128 pack b
lb bf16 681 72 64 aligned dw fast 256x128 split 2
lb bf16 41 1032 7232 aligned dw fast 256x192
lb bf16 65 1035 7813 odd dw fast 256x192 pack b
lb bf16 4075 136 8592 aligned dw fast 256x192 split 5
lb bf16 41 2056 5952 aligned dw fast 256x256
lb bf16 129 4949 2325 odd dw fast 256x256 pack b
lb bf16 2049 41 2031 odd dx any 128x128
lb bf16 65 925 5683 odd dx any 128x128 split 3
lb bf16 41 65 67 odd dx any 64x64
lb bf16 65 463 67 odd dx any 64x64 split 2
lb bf16 259 72 64 aligned dx fast 128x128
lb bf16 333 513 65 odd dx fast 128x128 pack b
lb bf16 264 840 64 aligned dx fast 128x128 split 3
lb bf16 3351 2049 65 odd dx fast 128x128 split 7 pack b
lb bf16 1032 48 6608 aligned dx fast 128x256
lb bf16 4911 333 3233 odd dx fast 128x256 pack b
lb bf16 41 1032 8248 aligned dx fast 128x256 split 4
lb bf16 2056 48 5544 aligned dx fast 192x256
lb bf16 1323 65 8079 odd dx fast 192x256 pack b
lb bf16 136 4392 8224 aligned dx fast 192x256 split 6
lb bf16 43 520 64 aligned dx fast 256x128
lb bf16 2049 605 1993 odd dx fast 256x128 pack b
lb bf16 72 688 64 aligned dx fast 256x128 split 2
lb bf16 1032 48 7232 aligned dx fast 256x192
lb bf16 1035 65 7813 odd dx fast 256x192 pack b
lb bf16 136 4080 8592 aligned dx fast 256x192 split 5
lb bf16 2056 48 5952 aligned dx fast 256x256
lb bf16 4949 129 2325 odd dx fast 256x256 pack b
lb f32 41 2049 2031 odd dw any 128x128
lb f32 613 65 8507 odd dw any 128x128 split 5
lb f32 41 201 8681 odd dw any 64x64
lb f32 41 200 8352 aligned dw fast 128x128
lb f32 65 199 8377 odd dw fast 128x128 pack b
lb f32 1091 72 5648 aligned dw fast 128x128 split 5
lb f32 771 65 5513 odd dw fast 128x128 split 5 pack b
lb f32 41 72 64 aligned dw fast 128x64
lb f32 41 65 67 odd dw fast 128x64 pack b
lb f32 293 72 64 aligned dw fast 128x64 split 2
lb f32 333 41 67 odd dw fast 128x64 split 2 pack b
lb f32 41 136 8248 aligned dw fast 64x128
lb f32 41 129 8319 odd dw fast 64x128 pack b
lb f32 520 48 4104 aligned dw fast 64x128 split 4
lb f32 1035 43 2315 odd dw fast 64x128 split 7 pack b
lb f32 2049 41 2031 odd dx any 128x128
lb f32 65 613 8507 odd dx any 128x128 split 5
lb f32 201 41 8681 odd dx any 64x64
lb f32 200 48 8224 aligned dx fast 128x128
lb f32 199 65 8377 odd dx fast 128x128 pack b
lb f32 67 1032 5776 aligned dx fast 128x128 split 5
lb f32 65 771 5513 odd dx fast 128x128 split 5 pack b
lb f32 41 72 64 aligned dx fast 128x64
lb f32 41 65 67 odd dx fast 128x64 pack b
lb f32 72 296 64 aligned dx fast 128x64 split 2
lb f32 41 333 67 odd dx fast 128x64 split 2 pack b
lb f32 136 48 8248 aligned dx fast 64x128
lb f32 129 41 8319 odd dx fast 64x128 pack b
lb f32 41 520 4160 aligned dx fast 64x128 split 4
lb f32 43 1035 2315 odd dx fast 64x128 split 7 pack b
linear bf16 451 8325 65 odd any 128x128
linear bf16 5459 67 1035 odd any 128x128 split 4
linear bf16 41 67 65 odd any 64x64
linear bf16 41 64 1032 aligned any 64x64 split 4
linear bf16 259 65 72 aligned fast 128x128
linear bf16 2699 207 1035 odd fast 128x128 pack
linear bf16 267 64 1032 aligned fast 128x128 split 4
linear bf16 937 861 2049 odd fast 128x128 split 3 pack
linear bf16 787 8281 72 aligned fast 128x256
linear bf16 41 8193 1032 aligned fast 128x256 split 4
linear bf16 1319 8273 72 aligned fast 192x256
linear bf16 2669 4441 65 odd fast 192x256 pack
linear bf16 43 65 520 aligned fast 256x128
linear bf16 1345 2953 1035 odd fast 256x128 pack
linear bf16 65 4129 1032 aligned fast 256x128 split 4
linear bf16 5409 1409 72 aligned fast 256x192
linear bf16 1695 4801 65 odd fast 256x192 pack
linear bf16 4955 2320 72 aligned fast 256x256
linear bf16 4949 2325 129 odd fast 256x256 pack
linear e4m3 451 8325 65 odd any 128x128
linear e4m3 5443 65 2049 odd any 128x128 split 4
linear e4m3 41 67 65 odd any 64x64
linear e4m3 41 71 1035 odd any 64x64 split 2
linear e4m3 41 64 272 aligned fast 128x128
linear e4m3 41 65 2064 aligned fast 128x128 split 4
linear e4m3 1319 8272 80 aligned fast 192x256
linear e4m3 4369 5629 65 odd fast 192x256 pack
linear e4m3 899 8481 80 aligned fast 256x192
linear e4m3 4739 6959 129 odd fast 256x192 pack
linear e4m3 4955 2320 80 aligned fast 256x256
linear e4m3 6549 8859 65 odd fast 256x256 pack
linear e4m3-fast 451 8325 65 odd any 128x128
linear e4m3-fast 5443 65 2049 odd any 128x128 split 4
linear e4m3-fast 41 67 65 odd any 64x64
linear e4m3-fast 41 71 1035 odd any 64x64 split 2
linear e4m3-fast 267 64 144 aligned fast 128x128
linear e4m3-fast 259 65 1035 odd fast 128x128 pack
linear e4m3-fast 259 64 2064 aligned fast 128x128 split 4
linear e4m3-fast 787 8281 80 aligned fast 128x256
linear e4m3-fast 41 8201 2064 aligned fast 128x256 split 4
linear e4m3-fast 1319 8272 80 aligned fast 192x256
linear e4m3-fast 1283 8375 129 odd fast 192x256 pack
linear e4m3-fast 41 64 272 aligned fast 256x128
linear e4m3-fast 5455 719 1035 odd fast 256x128 pack
linear e4m3-fast 41 65 2064 aligned fast 256x128 split 4
linear e4m3-fast 899 8480 80 aligned fast 256x192
linear e4m3-fast 1027 7785 129 odd fast 256x192 pack
linear e4m3-fast 4955 2321 80 aligned fast 256x256
linear e4m3-fast 4949 2325 129 odd fast 256x256 pack
linear f32 451 8325 65 odd any 128x128
linear f32 41 8475 1035 odd any 128x128 split 7
linear f32 405 8385 65 odd any 64x64
linear f32 197 8256 72 aligned fast 128x128
linear f32 199 8377 65 odd fast 128x128 pack
linear f32 5727 65 1032 aligned fast 128x128 split 5
linear f32 5459 67 1035 odd fast 128x128 split 5 pack
linear f32 41 64 72 aligned fast 128x64
linear f32 41 67 65 odd fast 128x64 pack
linear f32 43 64 520 aligned fast 128x64 split 4
linear f32 41 67 333 odd fast 128x64 split 2 pack
linear f32 137 8248 72 aligned fast 64x128
linear f32 129 8867 65 odd fast 64x128 pack
linear f32 41 4160 520 aligned fast 64x128 split 4
linear f32 43 2315 1035 odd fast 64x128 split 7 pack
"""


def cases():
    """(id, operator, type, e4m3's fast_sums, m, n, k, aligned, name)"""
    for line in LINES.strip().splitlines():
        op, kind, m, n, k, rows, name = line.split(" ", 6)
        yield (line.replace(" ", "-"), op, kind.split("-")[0], kind.endswith("fast"), int(m), int(n), int(k), rows == "aligned",
               name)


def planned(op, dtype, fast, m, n, k, aligned, out=None):
    """The library's name for a case's product, or its two."""
    code = {"f32": F32, "bf16": BF16, "e4m3": E4M3}[dtype]
    if op in ("linear", "gated"):
        out = out if out is not None else BF16 if dtype == "e4m3" else code
        f = mic.mic_gated_linear_forward_kernel_name if op == "gated" else mic.mic_linear_forward_kernel_name
        return f(None, code, out, fast, m, n, k, aligned).replace(" pack a pack b", " pack")
    if op == "gb":
        return mic.mic_gated_linear_backward_kernel_name(None, code, m, n, k, aligned)
    return mic.mic_linear_backward_kernel_name(None, code, mic.MIC_ACT_GELU if op == "lb" else mic.MIC_ACT_NONE, m, n, k, aligned)


def product_of(op, name, both):
    """The part of `both` that a case's name is about: forward's only one, dx's or dw's."""
    if op in ("linear", "gated"):
        return both
    dx, dw = both[len("dx: "):].split(", dw: ")
    return "dx " + dx if name.startswith("dx") else "dw " + dw
