/*
 * a4w4_binding.h -- the calls of a4w4.h that take many arguments, with those in an
 * array of 64-bit words instead: for bindings to whom each argument of a foreign
 * call has its price (Python's ctypes takes 0.15 to 0.25 us for one, 4 us for
 * a4w4_moe_route's seventeen; one packed argument takes 0.4).
 *
 * packed: the arguments of the call of the same name in its order, 8 bytes each, in
 * the machine's byte order, of any alignment: pointers and integers as 64-bit
 * integers, floats as doubles.  Copied before the call; same checks, same errors.
 */
#ifndef A4W4_BINDING_H_
#define A4W4_BINDING_H_

#ifdef __cplusplus
extern "C" {
#endif

int a4w4_packed_gemm_w8a8(const void* packed);        /* 11 words */
int a4w4_packed_kv_read(const void* packed);          /* 10 words */
int a4w4_packed_moe_route(const void* packed);        /* 17 words */
int a4w4_packed_qk_norm_rope(const void* packed);     /* 20 words */
int a4w4_packed_kv_append_rope(const void* packed);   /* 24 words */

#ifdef __cplusplus
}
#endif

#endif /* A4W4_BINDING_H_ */
